// lrm_route, lrm_route_backward, lrm_gate_dots: the router's softmax, its k choices, the balance
// loss and their gradient.
//
// "Expert Parallel Math Deep" (routing as an expectation over a batch; auxiliary loss): with
// p_te = softmax(l_t)_e, f_e the share of the pairs that go to expert e and P_e = mean_t p_te,
//   L_aux = coef E sum_e f_e P_e.
// f is piecewise constant in the logits, so with c = coef E / n
//   dL_aux/dl_te = c p_te (f_e - sum_e' f_e' p_te'),
// and the gate's gradient is a softmax backward of dL/dalpha, written in s_p = alpha_p dL/dalpha_p:
// over the k chosen logits s_j - alpha_j sum s, over all E logits [e chosen] s_j - p_te sum s.
// s_p itself is a row dot of the expert backward (lrm_gate_dots).
#include <math.h>

#include "lrm_device.hpp"
#include "lrm_forward.hpp"

namespace lrm {
namespace {

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kWave;

// Logits are ranked by one float64 key each: the float32 value is exact in float64 and leaves the
// low 29 mantissa bits zero, so the expert goes there (12 bits, E <= 4096), turned so that of two
// equal logits the lower expert has the larger key.  Every key of a row is distinct, and a maximum
// of keys is a maximum by (logit descending, expert ascending).  -0 becomes +0 first (they are
// equal logits); infinities, which hold no mantissa bits, and NaN move to +-2^200, beyond any
// float32: NaN ranks as -infinity.
constexpr double kKeyInf = 0x1p200;
constexpr double kNoKey = -0x1p300;   // below every key

__device__ __forceinline__ double route_key(float v, int e) {
  double d = (double)(v + 0.0f);
  d = fmin(fmax(d, -kKeyInf), kKeyInf);
  const int64_t b = __double_as_longlong(d);
  return __longlong_as_double(b | (b < 0 ? e : 4095 - e));
}

__device__ __forceinline__ int key_expert(double k) {
  const int64_t b = __double_as_longlong(k);
  const int low = (int)(b & 4095);
  return b < 0 ? low : 4095 - low;
}

// The key's logit (-infinity for NaN and -infinity).
__device__ __forceinline__ float key_logit(double k) {
  return (float)__longlong_as_double(__double_as_longlong(k) & ~(int64_t)4095);
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, kWave));
  return v;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

template <bool kBF16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  if (kBF16) return __uint_as_float((uint32_t)((const uint16_t*)row)[e] << 16);
  return ((const float*)row)[e];
}

// NaN or +infinity.
__device__ __forceinline__ bool bad_logit(float v) { return !(v < INFINITY); }

struct RouteArgs {
  const void* logits;
  const uint8_t* mask;
  int T, E, k, gate;
  int32_t* topk_idx;
  float* topk_w;
  float* lse;
  int32_t* part_tokens;  // [blocks][2]
  int32_t* part_counts;  // [blocks][E]
  float* part_prob;      // [blocks][E]
};

// One wavefront per token, any E and k: k rounds, each taking the largest key below the last one
// over the row (which stays in the caches).  The workgroup's waves keep sums of probabilities and
// counts of their own in LDS.
constexpr int kAnyWaves = 2;

template <bool kBF16>
__global__ __launch_bounds__(kAnyWaves * kWave) void route_any(RouteArgs a) {
  extern __shared__ float shared[];
  const int E = a.E, lane = lane_id(), w = threadIdx.x / kWave;
  float* prob = shared + w * E;                             // [waves][E]
  int* counts = (int*)(shared + kAnyWaves * E) + w * E;     // [waves][E]
  for (int e = lane; e < E; e += kWave) {
    prob[e] = 0.0f;
    counts[e] = 0;
  }
  int live = 0, bad = 0;
  const int nw = gridDim.x * kAnyWaves;
  for (int64_t t = (int64_t)blockIdx.x * kAnyWaves + w; t < a.T; t += nw) {
    const char* row = (const char*)a.logits + t * E * (kBF16 ? 2 : 4);
    double best = kNoKey;
    if (a.mask == nullptr || a.mask[t]) {
      for (int e = lane; e < E; e += kWave) {
        const float v = load_logit<kBF16>(row, e);
        if (bad_logit(v)) bad = LRM_DEVERR_NONFINITE;
        best = fmax(best, route_key(v, e));
      }
      best = wave_max(best);
    }
    const float m = key_logit(best);
    if (!(m > -INFINITY)) {   // masked, or no logit left
      for (int j = lane; j < a.k; j += kWave) {
        a.topk_idx[t * a.k + j] = -1;
        a.topk_w[t * a.k + j] = 0.0f;
      }
      if (lane == 0) a.lse[t] = 0.0f;
      continue;
    }
    ++live;
    float sum = 0.0f;
    for (int e = lane; e < E; e += kWave) sum += expf(key_logit(route_key(load_logit<kBF16>(row, e), e)) - m);
    sum = wave_sum_f32(sum);
    const float lse = m + logf(sum), inv = 1.0f / sum;
    if (lane == 0) a.lse[t] = lse;
    for (int e = lane; e < E; e += kWave)
      prob[e] += expf(key_logit(route_key(load_logit<kBF16>(row, e), e)) - m) * inv;
    float chosen = 0.0f;
    double key = best;
    for (int j = 0; j < a.k; ++j) {
      if (j > 0) {
        double next = kNoKey;
        for (int e = lane; e < E; e += kWave) {
          const double q = route_key(load_logit<kBF16>(row, e), e);
          next = q < key ? fmax(next, q) : next;
        }
        key = wave_max(next);
      }
      const float p = expf(key_logit(key) - m);
      chosen += p;
      if (lane == 0) {
        const int e = key_expert(key);
        a.topk_idx[t * a.k + j] = e;
        a.topk_w[t * a.k + j] = p;   // scaled below, by this lane
        ++counts[e];
      }
    }
    const float scale = a.gate == LRM_GATE_TOPK ? 1.0f / chosen : inv;
    if (lane == 0)
      for (int j = 0; j < a.k; ++j) a.topk_w[t * a.k + j] *= scale;
  }
  __shared__ int sh_live[kAnyWaves], sh_bad[kAnyWaves];
  const bool any_bad = ballot(bad != 0) != 0;
  if (lane == 0) {
    sh_live[w] = live;
    sh_bad[w] = any_bad ? LRM_DEVERR_NONFINITE : 0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kAnyWaves * kWave) {
    float p = 0.0f;
    int c = 0;
    for (int q = 0; q < kAnyWaves; ++q) {
      p += shared[q * E + e];
      c += ((int*)(shared + kAnyWaves * E))[q * E + e];
    }
    a.part_prob[(int64_t)blockIdx.x * E + e] = p;
    a.part_counts[(int64_t)blockIdx.x * E + e] = c;
  }
  if (threadIdx.x == 0) {
    int n = 0, b = 0;
    for (int q = 0; q < kAnyWaves; ++q) {
      n += sh_live[q];
      b |= sh_bad[q];
    }
    a.part_tokens[2 * blockIdx.x] = n;
    a.part_tokens[2 * blockIdx.x + 1] = b;
  }
}

// Sums the workgroups' partial results: counts, prob, the loss and the error word.  One workgroup
// of 1024 threads; thread (slice, e) adds every S-th workgroup's row in float64, then slice 0 adds
// the slices.
constexpr int kFinalThreads = 1024;

__global__ __launch_bounds__(kFinalThreads) void route_final(const int32_t* __restrict__ part_tokens,
                                                             const int32_t* __restrict__ part_counts,
                                                             const float* __restrict__ part_prob,
                                                             int blocks, int E, int k, float coef,
                                                             int32_t* __restrict__ counts,
                                                             float* __restrict__ prob,
                                                             float* __restrict__ loss,
                                                             int32_t* __restrict__ err) {
  __shared__ double sp[kFinalThreads];
  __shared__ int sc[kFinalThreads];
  __shared__ int tokens, bits;
  const int tid = threadIdx.x;
  if (tid == 0) tokens = bits = 0;
  __syncthreads();
  for (int b = tid; b < blocks; b += kFinalThreads) {
    atomicAdd(&tokens, part_tokens[2 * b]);
    atomicOr(&bits, part_tokens[2 * b + 1]);
  }
  __syncthreads();
  const int n = tokens;
  const int width = E >= kFinalThreads ? kFinalThreads : (E + kWave - 1) / kWave * kWave;
  const int S = kFinalThreads / width;
  const int slice = tid / width;
  double sum = 0.0;   // sum_e counts[e] * (sum of p_te)
  for (int e0 = 0; e0 < E; e0 += width) {
    const int e = e0 + tid % width;
    double p = 0.0;
    int c = 0;
    if (e < E && slice < S)
      for (int b = slice; b < blocks; b += S) {
        p += part_prob[(int64_t)b * E + e];
        c += part_counts[(int64_t)b * E + e];
      }
    sp[tid] = p;
    sc[tid] = c;
    __syncthreads();
    if (slice == 0 && e < E) {
      for (int q = 1; q < S; ++q) {
        p += sp[tid + q * width];
        c += sc[tid + q * width];
      }
      counts[e] = c;
      prob[e] = n > 0 ? (float)(p / n) : 0.0f;
      sum += p * c;
    }
    __syncthreads();
  }
  sp[tid] = sum;
  __syncthreads();
  for (int o = kFinalThreads / 2; o >= 1; o >>= 1) {
    if (tid < o) sp[tid] += sp[tid + o];
    __syncthreads();
  }
  if (tid == 0) {
    const double nn = n;
    *loss = n > 0 ? (float)((double)coef * E * sp[0] / (nn * nn * k)) : 0.0f;
    *err = bits;
  }
}

// dlogits: one wavefront per token, passes over the row for its maximum, its sums and the output
// (all but the first from the caches).
template <bool kBF16>
__global__ __launch_bounds__(kBlock) void route_backward(const void* __restrict__ logits,
                                                         const int32_t* __restrict__ topk_idx,
                                                         const float* __restrict__ topk_w,
                                                         const int32_t* __restrict__ counts,
                                                         const float* __restrict__ adot, int T,
                                                         int E, int k, int gate, float coef,
                                                         float* __restrict__ dlogits) {
  const int lane = lane_id();
  int pairs = 0;
  for (int e = lane; e < E; e += kWave) pairs += counts[e];
  pairs = wave_sum_int(pairs);
  // f_e = counts[e] / (n k) and c = coef E / n with n = pairs / k
  const float f1 = pairs > 0 ? 1.0f / (float)pairs : 0.0f;
  const float c = pairs > 0 ? (float)((double)coef * E * k / pairs) : 0.0f;
  const int64_t nw = (int64_t)gridDim.x * kWavesPerBlock;
  for (int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; t < T; t += nw) {
    const char* row = (const char*)logits + t * E * (kBF16 ? 2 : 4);
    float* out = dlogits + t * E;
    if (topk_idx[t * k] < 0) {
      for (int e = lane; e < E; e += kWave) out[e] = 0.0f;
      continue;
    }
    float m = -INFINITY;
    for (int e = lane; e < E; e += kWave) m = fmaxf(m, load_logit<kBF16>(row, e));
    m = wave_max_f32(m);
    float sum = 0.0f, fp = 0.0f;
    for (int e = lane; e < E; e += kWave) {
      const float p = expf(load_logit<kBF16>(row, e) - m);
      sum += p;
      fp += f1 * counts[e] * p;
    }
    const float inv = 1.0f / wave_sum_f32(sum);
    fp = wave_sum_f32(fp) * inv;
    float S = 0.0f;
    if (adot != nullptr)
      for (int j = 0; j < k; ++j) S += adot[t * k + j];
    const float all = gate == LRM_GATE_ALL ? S : 0.0f;
    for (int e = lane; e < E; e += kWave) {
      const float p = expf(load_logit<kBF16>(row, e) - m) * inv;
      float g = p * (c * (f1 * counts[e] - fp) - all);
      if (adot != nullptr)
        for (int j = 0; j < k; ++j)
          if (topk_idx[t * k + j] == e)
            g += adot[t * k + j] - (gate == LRM_GATE_TOPK ? topk_w[t * k + j] * S : 0.0f);
      out[e] = g;
    }
  }
}

// adot = 0 everywhere, and the pair -> compacted-row map of the retained rows.
__global__ __launch_bounds__(kBlock) void gate_rows(const int32_t* __restrict__ sel_pair,
                                                    const int32_t* __restrict__ cmp_off, int E_loc,
                                                    int K_cap, int64_t P, int32_t* __restrict__ map,
                                                    float* __restrict__ adot,
                                                    int32_t* __restrict__ err) {
  int K = cmp_off[E_loc];
  K = K < 0 ? 0 : (K > K_cap ? K_cap : K);
  const int64_t n = (int64_t)gridDim.x * kBlock;
  for (int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x; i < P || i < K; i += n) {
    if (i < P) adot[i] = 0.0f;
    if (i < K) {
      const int p = sel_pair[i];
      if (p >= 0 && p < P)
        map[p] = (int32_t)i;
      else
        set_error(err, LRM_DEVERR_INDEX);
    }
  }
}

// adot[sel_pair[i]] = <dphi[i], Phic[i]>: 16 lanes per retained row, float64 sums in a fixed order.
// Memory-bound: 4 + (2 or 4) bytes per multiplied pair of elements.
constexpr int kLanesPerRow = 16;
constexpr int kRowsPerWave = kWave / kLanesPerRow;

template <bool kBF16>
__global__ __launch_bounds__(kBlock) void gate_dots(const int32_t* __restrict__ sel_pair,
                                                    const int32_t* __restrict__ cmp_off, int E_loc,
                                                    int K_cap, int64_t P, int d,
                                                    const float* __restrict__ dphi,
                                                    const void* __restrict__ Phic,
                                                    const int32_t* __restrict__ map,
                                                    float* __restrict__ adot,
                                                    int32_t* __restrict__ err) {
  int K = cmp_off[E_loc];
  K = K < 0 ? 0 : (K > K_cap ? K_cap : K);
  const int lane = lane_id(), sub = lane % kLanesPerRow;
  const int64_t groups = ((int64_t)K + kRowsPerWave - 1) / kRowsPerWave;
  const int64_t nw = (int64_t)gridDim.x * kWavesPerBlock;
  for (int64_t gi = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; gi < groups; gi += nw) {
    const int64_t i = gi * kRowsPerWave + lane / kLanesPerRow;
    const bool live = i < K;
    const float* g = dphi + (live ? i : 0) * d;
    const char* f = (const char*)Phic + (live ? i : 0) * d * (kBF16 ? 2 : 4);
    double acc = 0.0;
    for (int c = sub; c < d / 4; c += kLanesPerRow) {
      const float4 v = load_nt((const float4*)g + c);
      float u0, u1, u2, u3;
      if (kBF16) {
        const uint2 w = ((const uint2*)f)[c];
        u0 = bf16_lo(w.x);
        u1 = bf16_hi(w.x);
        u2 = bf16_lo(w.y);
        u3 = bf16_hi(w.y);
      } else {
        const float4 w = load_nt((const float4*)f + c);
        u0 = w.x;
        u1 = w.y;
        u2 = w.z;
        u3 = w.w;
      }
      acc += (double)v.x * u0;
      acc += (double)v.y * u1;
      acc += (double)v.z * u2;
      acc += (double)v.w * u3;
    }
#pragma unroll
    for (int o = kLanesPerRow / 2; o >= 1; o >>= 1) acc += __shfl_xor(acc, o, kWave);
    if (live && sub == 0) {
      const int p = sel_pair[i];
      if (p >= 0 && p < P) {
        if (map[p] == i)
          adot[p] = (float)acc;
        else
          set_error(err, LRM_DEVERR_INDEX);   // another row names this pair
      }
    }
  }
}

unsigned grid_for(int64_t blocks, unsigned cap) {
  return (unsigned)(blocks < 1 ? 1 : (blocks < cap ? blocks : cap));
}

}  // namespace

hipError_t launch_route(const lrm_router& r, const void* logits, const uint8_t* mask,
                        int32_t* topk_idx, float* topk_w, float* lse, int32_t* counts, float* prob,
                        float* loss, char* ws, hipStream_t s) {
  const RouteWs wl = route_ws(r.E);
  RouteArgs a{logits, mask, r.T, r.E, r.k, r.gate, topk_idx, topk_w, lse,
              (int32_t*)(ws + wl.tokens), (int32_t*)(ws + wl.counts), (float*)(ws + wl.prob)};
  const unsigned nb = grid_for(((int64_t)r.T + kAnyWaves - 1) / kAnyWaves, kRouteBlocks);
  const size_t lds = (size_t)kAnyWaves * r.E * 8;
  if (r.dtype == LRM_BF16)
    hipLaunchKernelGGL(route_any<true>, dim3(nb), dim3(kAnyWaves * kWave), lds, s, a);
  else
    hipLaunchKernelGGL(route_any<false>, dim3(nb), dim3(kAnyWaves * kWave), lds, s, a);
  hipLaunchKernelGGL(route_final, dim3(1), dim3(kFinalThreads), 0, s, a.part_tokens, a.part_counts,
                     a.part_prob, (int)nb, r.E, r.k, r.balance_coef, counts, prob, loss,
                     (int32_t*)(ws + wl.err));
  return hipGetLastError();
}

hipError_t launch_route_backward(const lrm_router& r, const void* logits, const int32_t* topk_idx,
                                 const float* topk_w, const int32_t* counts,
                                 const float* adot, float* dlogits, hipStream_t s) {
  const unsigned nb = grid_for(((int64_t)r.T + kWavesPerBlock - 1) / kWavesPerBlock, 4096);
  if (r.dtype == LRM_BF16)
    hipLaunchKernelGGL(route_backward<true>, dim3(nb), dim3(kBlock), 0, s, logits, topk_idx, topk_w,
                       counts, adot, r.T, r.E, r.k, r.gate, r.balance_coef, dlogits);
  else
    hipLaunchKernelGGL(route_backward<false>, dim3(nb), dim3(kBlock), 0, s, logits, topk_idx, topk_w,
                       counts, adot, r.T, r.E, r.k, r.gate, r.balance_coef, dlogits);
  return hipGetLastError();
}

hipError_t launch_gate_dots(const lrm_problem& p, const int32_t* sel_pair, const int32_t* cmp_off,
                            const float* dphi, const void* Phic, float* adot, char* ws,
                            hipStream_t s) {
  int32_t* err = (int32_t*)ws;
  int32_t* map = (int32_t*)(ws + kForwardMap);
  const int64_t P = (int64_t)p.T * p.k;
  const int64_t most = P > p.K_cap ? P : p.K_cap;
  hipLaunchKernelGGL(gate_rows, dim3(grid_for((most + kBlock - 1) / kBlock, 2048)), dim3(kBlock), 0,
                     s, sel_pair, cmp_off, p.E_loc, p.K_cap, P, map, adot, err);
  const int64_t rows = ((int64_t)p.K_cap + kRowsPerWave * kWavesPerBlock - 1) / (kRowsPerWave * kWavesPerBlock);
  const unsigned nb = grid_for(rows, 4096);
  if (p.dtype == LRM_BF16)
    hipLaunchKernelGGL(gate_dots<true>, dim3(nb), dim3(kBlock), 0, s, sel_pair, cmp_off, p.E_loc,
                       p.K_cap, P, p.d, dphi, Phic, map, adot, err);
  else
    hipLaunchKernelGGL(gate_dots<false>, dim3(nb), dim3(kBlock), 0, s, sel_pair, cmp_off, p.E_loc,
                       p.K_cap, P, p.d, dphi, Phic, map, adot, err);
  return hipGetLastError();
}

}  // namespace lrm
