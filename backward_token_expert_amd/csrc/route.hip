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

__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

__device__ __forceinline__ double route_key(float v, int e) {
  const double d = min64(max64((double)(v + 0.0f), -kKeyInf), kKeyInf);   // NaN: the other operand
  const int hi = __double2hiint(d);
  return __hiloint2double(hi, __double2loint(d) | ((e ^ 4095) ^ ((hi >> 31) & 4095)));
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
  int pitch;             // E rounded up to 4
  int32_t* part_counts;  // [blocks][pitch], columns past E are 0
  float* part_prob;      // [blocks][pitch]
};

// One wavefront per token, any E and k: k rounds, each taking the largest key below the last one
// over the row (which stays in the caches).  The workgroup's waves keep sums of probabilities of
// their own, and counts together, in LDS.
constexpr int kAnyWaves = 2;

template <bool kBF16>
__global__ __launch_bounds__(kAnyWaves * kWave) void route_any(RouteArgs a) {
  extern __shared__ float shared[];
  const int E = a.E, lane = lane_id(), w = threadIdx.x / kWave;
  float* prob = shared + w * E;                     // [waves][E]
  int* counts = (int*)(shared + kAnyWaves * E);     // [E]
  for (int e = lane; e < E; e += kWave) prob[e] = 0.0f;
  for (int e = threadIdx.x; e < E; e += kAnyWaves * kWave) counts[e] = 0;
  __syncthreads();
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
        atomicAdd(&counts[e], 1);
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
  for (int e = threadIdx.x; e < a.pitch; e += kAnyWaves * kWave) {
    float p = 0.0f;
    for (int q = 0; q < kAnyWaves && e < E; ++q) p += shared[q * E + e];
    a.part_prob[(int64_t)blockIdx.x * a.pitch + e] = p;
    a.part_counts[(int64_t)blockIdx.x * a.pitch + e] = e < E ? counts[e] : 0;
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

// Registers-only routing for k <= KT and E <= LPT * VPL: LPT adjacent lanes share a token, each
// holding up to VPL logits in 16-byte chunks (chunk i * LPT + sub, so a token's lanes read 16 LPT
// consecutive bytes).  Each lane sorts its keys in groups of KT (an odd-even merge network; a
// comparator is one float64 maximum and one minimum) and merges every group into the KT largest so
// far (maximum of one list against the other reversed, then a bitonic sort); log2(LPT) merges
// across lanes leave the token's list in all of them.  For KT = 8 that is 9 instructions a logit,
// where inserting each key into the list takes 16, and the comparators of a stage do not wait for
// each other.  Few lanes a token keep the wave's work in the sorting of distinct logits rather
// than in the merges that every lane repeats.
// The value of a lane of the other half of each group of 2 * O lanes (all lanes of a half hold the
// same value when O > 1 and O < 16, so a mirror serves as the exchange).
template <int O>
__device__ __forceinline__ int swap_half(int v) {
  if constexpr (O == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);        // 1 0 3 2
  else if constexpr (O == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // 2 3 0 1
  else if constexpr (O == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // mirror of 8
  else if constexpr (O == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // mirror of 16
  else return __shfl_xor(v, O, kWave);
}
template <int O>
__device__ __forceinline__ float swap_half(float v) {
  return __int_as_float(swap_half<O>(__float_as_int(v)));
}
template <int O>
__device__ __forceinline__ double swap_half(double v) {
  return __hiloint2double(swap_half<O>(__double2hiint(v)), swap_half<O>(__double2loint(v)));
}

// Sum or maximum over a token's LPT lanes, in all of them.
template <int LPT, int O = 1>
__device__ __forceinline__ float token_sum(float v) {
  if constexpr (O < LPT) return token_sum<LPT, 2 * O>(v + swap_half<O>(v));
  return v;
}
template <int LPT, int O = 1>
__device__ __forceinline__ float token_max(float v) {
  if constexpr (O < LPT) return token_max<LPT, 2 * O>(fmaxf(v, swap_half<O>(v)));
  return v;
}

// Descending sort of N keys in registers: Batcher's odd-even merge network.
template <int N>
__device__ __forceinline__ void sort_keys(double (&t)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const double a = t[i + j], b = t[i + j + k];
            t[i + j] = max64(a, b);
            t[i + j + k] = min64(a, b);
          }
}

// t, sorted, becomes the N largest of t and the sorted list whose reverse is r.
template <int N>
__device__ __forceinline__ void merge_keys(double (&t)[N], const double (&r)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = max64(t[j], r[j]);
#pragma unroll
  for (int s = N / 2; s >= 1; s /= 2)
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!(j & s)) {
        const double a = t[j], b = t[j + s];
        t[j] = max64(a, b);
        t[j + s] = min64(a, b);
      }
}

template <int KT, int LPT, int O = 1>
__device__ __forceinline__ void merge_lanes(double (&t)[KT]) {
  if constexpr (O < LPT) {
    double r[KT];
#pragma unroll
    for (int j = 0; j < KT; ++j) r[j] = swap_half<O>(t[KT - 1 - j]);
    merge_keys(t, r);
    merge_lanes<KT, LPT, 2 * O>(t);
  }
}

// exp(v - m) for v <= m by the hardware's power of two.  The argument's two roundings and the constant's
// put it off by at most 2.3 (m - v) 2^-24 of itself, the instruction by 2 2^-24 more: in all less than 3
// 2^-24 of the row's largest, which is what the sum and the weights' sum to 1 rest on.
__device__ __forceinline__ float exp_below(float v, float m) {
  return __builtin_amdgcn_exp2f((v - m) * 1.44269504f);
}

// A lane's logits of one row: VPL values, -infinity past E or where the row is not wanted.  `vec`:
// rows are multiples of 16 bytes.
template <bool kBF16, int LPT, int VPL>
__device__ __forceinline__ void load_row(const char* row, int E, int sub, bool want, bool vec,
                                         float (&v)[VPL]) {
  constexpr int CV = kBF16 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < VPL / CV; ++i) {
    const int e0 = (i * LPT + sub) * CV;
#pragma unroll
    for (int q = 0; q < CV; ++q) v[i * CV + q] = -INFINITY;
    if (i * LPT * CV >= E) continue;   // uniform
    if (vec) {
      if (want && e0 < E) {
        const uint4 x = ((const uint4*)row)[i * LPT + sub];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (kBF16) {
            v[i * CV + 2 * q] = bf16_lo(w[q]);
            v[i * CV + 2 * q + 1] = bf16_hi(w[q]);
          } else {
            v[i * CV + q] = __uint_as_float(w[q]);
          }
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < CV; ++q)
        if (want && e0 + q < E) v[i * CV + q] = load_logit<kBF16>(row, e0 + q);
    }
  }
}

struct RouteOut {
  int32_t* counts;
  float* prob;
  float* loss;
  int32_t* err;
  float coef;
};

template <bool kBF16, int LPT, int VPL, int KT, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void route_rows(RouteArgs a, RouteOut o, int vec) {
  constexpr int CV = kBF16 ? 8 : 4, TPW = kWave / LPT;
  constexpr int ROWS = LPT <= 16 ? 4 : 1;   // partial sums of a wave: one per 16 lanes, or one
  constexpr int THREADS = WAVES * kWave;
  extern __shared__ float shared[];
  const int E = a.E, lane = lane_id(), w = threadIdx.x / kWave, sub = lane % LPT;
  float* part = shared;                            // [WAVES * ROWS][E]
  int* counts = (int*)(shared + WAVES * ROWS * E); // [E]
  __shared__ int live_sum, bits;
  for (int e = threadIdx.x; e < E; e += THREADS) counts[e] = 0;
  if (threadIdx.x == 0) live_sum = bits = 0;
  __syncthreads();
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  int live = 0, bad = 0;
  const int64_t step = (int64_t)gridDim.x * WAVES * TPW;
  for (int64_t t0 = ((int64_t)blockIdx.x * WAVES + w) * TPW; t0 < a.T; t0 += step) {
    const int64_t t = t0 + lane / LPT;
    const bool want = t < a.T && (a.mask == nullptr || a.mask[t]);
    float v[VPL];
    load_row<kBF16, LPT, VPL>((const char*)a.logits + (want ? t : 0) * E * (kBF16 ? 2 : 4), E, sub,
                              want, vec, v);
    double key[KT];
#pragma unroll
    for (int i0 = 0; i0 < VPL; i0 += KT) {
      if (i0 / CV * LPT * CV >= E) continue;   // uniform
      double group[KT];
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        const int i = i0 + j, e = (i / CV * LPT + sub) * CV + i % CV;
        group[j] = e < E ? route_key(v[i], e) : kNoKey;
      }
      sort_keys(group);
      if (i0 == 0) {
#pragma unroll
        for (int j = 0; j < KT; ++j) key[j] = group[j];
      } else {
        double r[KT];
#pragma unroll
        for (int j = 0; j < KT; ++j) r[j] = group[KT - 1 - j];
        merge_keys(key, r);
      }
    }
    merge_lanes<KT, LPT>(key);
    const float top = key_logit(key[0]);
    const bool ok = want && top > -INFINITY;
    const float m = ok ? top : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i / CV * LPT * CV >= E) continue;
      v[i] = exp_below(v[i], m);
      sum += v[i];
    }
    sum = token_sum<LPT>(sum);
    if (!(sum < INFINITY)) bad = LRM_DEVERR_NONFINITE;   // a NaN, or infinity less itself
    const float inv = ok ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i / CV * LPT * CV >= E) continue;
      acc[i] += v[i] * inv;
    }
    float p[KT], chosen = 0.0f;
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      p[j] = exp_below(key_logit(key[j]), m);
      chosen += j < a.k ? p[j] : 0.0f;
    }
    const float scale = a.gate == LRM_GATE_TOPK ? (ok ? 1.0f / chosen : 0.0f) : inv;
    if (t < a.T) {
      if (sub == 0) {
        a.lse[t] = ok ? m + __logf(sum) : 0.0f;
        live += ok;
      }
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (j % LPT == sub && j < a.k) {
          const int e = ok ? key_expert(key[j]) : -1;
          a.topk_idx[t * a.k + j] = e;
          a.topk_w[t * a.k + j] = p[j] * scale;
          if (e >= 0) atomicAdd(&counts[e], 1);
        }
    }
  }
  // over the tokens of a wave: lanes of one sub within 16 lanes by rotations, the rest in LDS
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (i / CV * LPT * CV >= E) continue;
    float x = acc[i];
    if constexpr (LPT <= 4) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x124, 0xF, 0xF, true));
    if constexpr (LPT <= 8) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x128, 0xF, 0xF, true));
    const int e = (i / CV * LPT + sub) * CV + i % CV;
    if ((LPT > 16 || lane % 16 < LPT) && e < E) part[(w * ROWS + (ROWS > 1 ? lane / 16 : 0)) * E + e] = x;
  }
  live = wave_sum_int(live);
  const bool any_bad = ballot(bad != 0) != 0;
  if (lane == 0) {
    atomicAdd(&live_sum, live);
    if (any_bad) atomicOr(&bits, LRM_DEVERR_NONFINITE);
  }
  __syncthreads();
  const int n = live_sum;
  double mine = 0.0;   // of sum_e counts[e] * (sum of p_te), where this workgroup is the only one
  for (int e = threadIdx.x; e < (gridDim.x > 1 ? a.pitch : E); e += THREADS) {
    float x = 0.0f;
    if (e < E) {
#pragma unroll 8
      for (int q = 0; q < WAVES * ROWS; ++q) x += part[q * E + e];
    }
    if (gridDim.x > 1) {
      a.part_prob[(int64_t)blockIdx.x * a.pitch + e] = x;
      a.part_counts[(int64_t)blockIdx.x * a.pitch + e] = e < E ? counts[e] : 0;
    } else {
      o.counts[e] = counts[e];
      o.prob[e] = n > 0 ? (float)((double)x / n) : 0.0f;
      mine += (double)x * counts[e];
    }
  }
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      a.part_tokens[2 * blockIdx.x] = n;
      a.part_tokens[2 * blockIdx.x + 1] = bits;
    }
    return;
  }
  __shared__ double sums[WAVES];
  mine = wave_sum(mine);
  if (lane == 0) sums[w] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double x = 0.0;
    for (int q = 0; q < WAVES; ++q) x += sums[q];
    const double nn = n;
    *o.loss = n > 0 ? (float)((double)o.coef * E * x / (nn * nn * a.k)) : 0.0f;
    *o.err = bits;
  }
}

// Sums the workgroups' partial results: counts, prob, the loss and the error word.  One workgroup;
// thread (slice, q) adds four experts' columns of every S-th workgroup's row in float64, kBatch rows
// in flight (one after the other the rows' latencies were all of this kernel's time: 17 us for 256
// rows of 128 experts), then the slices are added in order.
constexpr int kFinalThreads = 1024, kBatch = 8;

__global__ __launch_bounds__(kFinalThreads) void route_final(const int32_t* __restrict__ part_tokens,
                                                             const int32_t* __restrict__ part_counts,
                                                             const float* __restrict__ part_prob,
                                                             int blocks, int E, int pitch, int k,
                                                             float coef, int32_t* __restrict__ counts,
                                                             float* __restrict__ prob,
                                                             float* __restrict__ loss,
                                                             int32_t* __restrict__ err) {
  __shared__ double sp[kFinalThreads][4];
  __shared__ int sc[kFinalThreads][4];
  __shared__ double sums[kFinalThreads / kWave];
  __shared__ int tokens, bits;
  const int tid = threadIdx.x, Q = pitch / 4, S = kFinalThreads / Q;   // pitch <= 4096
  const int slice = tid / Q, q = tid % Q;
  if (tid == 0) tokens = bits = 0;
  int n = 0, bad = 0;
  for (int b = tid; b < blocks; b += kFinalThreads) {
    const int2 x = ((const int2*)part_tokens)[b];
    n += x.x;
    bad |= x.y;
  }
  double p[4] = {0.0, 0.0, 0.0, 0.0};
  int c[4] = {0, 0, 0, 0};
  if (slice < S)
    for (int b0 = slice; b0 < blocks; b0 += kBatch * S) {
      float4 x[kBatch];
      int4 y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int b = b0 + i * S;
        x[i] = b < blocks ? ((const float4*)(part_prob + (int64_t)b * pitch))[q] : make_float4(0, 0, 0, 0);
        y[i] = b < blocks ? ((const int4*)(part_counts + (int64_t)b * pitch))[q] : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        p[0] += x[i].x;
        p[1] += x[i].y;
        p[2] += x[i].z;
        p[3] += x[i].w;
        c[0] += y[i].x;
        c[1] += y[i].y;
        c[2] += y[i].z;
        c[3] += y[i].w;
      }
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sp[tid][i] = p[i];
    sc[tid][i] = c[i];
  }
  __syncthreads();
  n = wave_sum_int(n);
  bad = ballot(bad != 0) != 0 ? LRM_DEVERR_NONFINITE : 0;
  if (lane_id() == 0) {
    atomicAdd(&tokens, n);
    atomicOr(&bits, bad);
  }
  __syncthreads();
  n = tokens;
  double sum = 0.0;   // sum_e counts[e] * (sum of p_te)
  for (int e = tid; e < E; e += kFinalThreads) {
    double x = 0.0;
    int y = 0;
#pragma unroll 8
    for (int i = 0; i < S; ++i) {
      x += sp[i * Q + e / 4][e % 4];
      y += sc[i * Q + e / 4][e % 4];
    }
    counts[e] = y;
    prob[e] = n > 0 ? (float)(x / n) : 0.0f;
    sum += x * y;
  }
  sum = wave_sum(sum);
  if (lane_id() == 0) sums[tid / kWave] = sum;
  __syncthreads();
  if (tid == 0) {
    double x = 0.0;
    for (int i = 0; i < kFinalThreads / kWave; ++i) x += sums[i];
    const double nn = n;
    *loss = n > 0 ? (float)((double)coef * E * x / (nn * nn * k)) : 0.0f;
    *err = bits;
  }
}

// dlogits, with the lanes and registers of route_rows.  The gate's terms on the k chosen experts
// go through a row of zeros in LDS, where their lanes of the row pick them up; a lane's own
// register for an expert is not indexable.
template <bool kBF16, int LPT, int VPL, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void route_backward(const void* __restrict__ logits,
                                                                const int32_t* __restrict__ topk_idx,
                                                                const float* __restrict__ topk_w,
                                                                const int32_t* __restrict__ counts,
                                                                const float* __restrict__ adot,
                                                                int T, int E, int k, int gate,
                                                                float coef, int vec,
                                                                float* __restrict__ dlogits) {
  constexpr int CV = kBF16 ? 8 : 4, TPW = kWave / LPT;
  constexpr int G = LPT >= 8 ? 1 : 8 / LPT;   // choices a lane has in registers
  extern __shared__ float shared[];
  const int lane = lane_id(), w = threadIdx.x / kWave, sub = lane % LPT;
  float* extra = shared + (w * TPW + lane / LPT) * E;   // this token's row
  int pairs = 0;
  for (int e = lane; e < E; e += kWave) pairs += counts[e];
  int n[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = (i / CV * LPT + sub) * CV + i % CV;
    n[i] = e < E ? counts[e] : 0;
    if (adot != nullptr && e < E) extra[e] = 0.0f;
  }
  float f[VPL], c = 0.0f;
  bool first = true;
  const bool vec_out = E % 4 == 0;
  const int64_t step = (int64_t)gridDim.x * WAVES * TPW;
  for (int64_t t0 = ((int64_t)blockIdx.x * WAVES + w) * TPW; t0 < T; t0 += step) {
    const int64_t t = t0 + lane / LPT;
    const bool in = t < T;
    // every load of the token at once: the row (also of a token that turns out not to be valid), its
    // choices and their terms
    float v[VPL];
    load_row<kBF16, LPT, VPL>((const char*)logits + (in ? t : 0) * E * (kBF16 ? 2 : 4), E, sub, in, vec, v);
    int ge[G];
    float ga[G], gw[G];
#pragma unroll
    for (int q = 0; q < G; ++q) {
      const int j = sub + q * LPT;
      const bool has = in && adot != nullptr && j < k;
      ge[q] = has ? topk_idx[t * k + j] : -1;
      ga[q] = has ? adot[t * k + j] : 0.0f;
      gw[q] = has && gate == LRM_GATE_TOPK ? topk_w[t * k + j] : 0.0f;
    }
    const bool ok = in && topk_idx[t * k] >= 0;
    if (first) {
      // f_e = counts[e] / (n k) and c = coef E / n with n = pairs / k
      pairs = wave_sum_int(pairs);
      const float f1 = pairs > 0 ? 1.0f / (float)pairs : 0.0f;
      c = pairs > 0 ? (float)((double)coef * E * k / pairs) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) f[i] = f1 * n[i];
      first = false;
    }
    float S = 0.0f;
    if (adot != nullptr) {
#pragma unroll
      for (int q = 0; q < G; ++q) S += ga[q];
      if (in)
        for (int j = sub + G * LPT; j < k; j += LPT) S += adot[t * k + j];
      S = token_sum<LPT>(S);
      S = ok ? S : 0.0f;
      if (ok) {
#pragma unroll
        for (int q = 0; q < G; ++q)
          if (ge[q] >= 0 && ge[q] < E) atomicAdd(&extra[ge[q]], ga[q] - gw[q] * S);
        for (int j = sub + G * LPT; j < k; j += LPT) {
          const int e = topk_idx[t * k + j];
          const float x = adot[t * k + j] - (gate == LRM_GATE_TOPK ? topk_w[t * k + j] * S : 0.0f);
          if (e >= 0 && e < E) atomicAdd(&extra[e], x);
        }
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i / CV * LPT * CV >= E) continue;
      m = fmaxf(m, v[i]);
    }
    m = token_max<LPT>(m);
    m = ok ? m : 0.0f;
    float sum = 0.0f, fp = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (i / CV * LPT * CV >= E) continue;
      v[i] = exp_below(v[i], m);
      sum += v[i];
      fp += f[i] * v[i];
    }
    const float inv = ok ? 1.0f / token_sum<LPT>(sum) : 0.0f;
    fp = token_sum<LPT>(fp) * inv;
    const float all = gate == LRM_GATE_ALL ? S : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in) {
#pragma unroll
      for (int i = 0; i < VPL / 4; ++i) {
        const int e0 = (i * 4 / CV * LPT + sub) * CV + i * 4 % CV;
        if (i * 4 / CV * LPT * CV >= E) continue;
        float g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          g[q] = ok ? v[4 * i + q] * inv * (c * (f[4 * i + q] - fp) - all) : 0.0f;
          if (adot != nullptr && e0 + q < E) g[q] += extra[e0 + q];
        }
        float* out = dlogits + t * E + e0;
        if (vec_out) {
          if (e0 < E) *(float4*)out = make_float4(g[0], g[1], g[2], g[3]);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (e0 + q < E) out[q] = g[q];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (adot != nullptr && ok) {
#pragma unroll
      for (int q = 0; q < G; ++q)
        if (ge[q] >= 0 && ge[q] < E) extra[ge[q]] = 0.0f;
      for (int j = sub + G * LPT; j < k; j += LPT) {
        const int e = topk_idx[t * k + j];
        if (e >= 0 && e < E) extra[e] = 0.0f;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
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

namespace {

template <bool kBF16, int LPT, int VPL, int KT, int WAVES>
unsigned launch_rows(const RouteArgs& a, const RouteOut& o, hipStream_t s) {
  constexpr int kTokens = WAVES * kWave / LPT, kRows = LPT <= 16 ? 4 : 1;
  const unsigned nb = grid_for(((int64_t)a.T + kTokens - 1) / kTokens, kRouteBlocks);
  const size_t lds = (size_t)(WAVES * kRows + 1) * a.E * 4;
  const int vec = (int64_t)a.E * (kBF16 ? 2 : 4) % 16 == 0;
  hipLaunchKernelGGL((route_rows<kBF16, LPT, VPL, KT, WAVES>), dim3(nb), dim3(WAVES * kWave), lds, s,
                     a, o, vec);
  return nb;
}

// Up to this many tokens (one pass of 256 workgroups) the shapes with more lanes a token.  Router /
// gradient in us, E 128, k 8, f32, with 16 lanes against 8: 256 tokens 10.0 / 4.6 against 14.0 / 6.8; 4096
// 11.4 / 4.8 against 14.8 / 7.1; 8192 12.5 / 5.6 against 15.1 / 7.4; 16384 15.2 / 7.4 against 15.9 / 8.6, with
// bf16 logits 14.8 / 8.9 against 15.1 / 8.2; 32768 21.9 / 15.9 against 19.4 / 14.0.
constexpr int kShortBatch = 8192;

template <bool kBF16, int KT>
unsigned launch_rows_e(const RouteArgs& a, const RouteOut& o, hipStream_t s) {
  // few tokens: more lanes each, for the latency of one token's chain (one token 10.4 us with 4
  // lanes, 7.2 with 8, 5.8 with 16)
  if (a.E <= 128 && a.T <= kShortBatch) return launch_rows<kBF16, 16, 8, KT, 8>(a, o, s);
  if (a.E <= 128) return launch_rows<kBF16, 8, 16, KT, 16>(a, o, s);
  if (a.E <= 256) return launch_rows<kBF16, 8, 32, KT, 8>(a, o, s);
  if (a.E <= 512) return launch_rows<kBF16, 16, 32, KT, 4>(a, o, s);
  return launch_rows<kBF16, 64, 64, KT, 2>(a, o, s);
}

template <bool kBF16>
unsigned launch_rows_any(const RouteArgs& a, const RouteOut& o, hipStream_t s) {
  if (a.k <= 2) return launch_rows_e<kBF16, 2>(a, o, s);
  if (a.k <= 8) return launch_rows_e<kBF16, 8>(a, o, s);
  if (a.k <= 16) return launch_rows_e<kBF16, 16>(a, o, s);
  // more choices than a lane's registers sort: a round of maxima per choice
  const unsigned nb = grid_for(((int64_t)a.T + kAnyWaves - 1) / kAnyWaves, kRouteBlocks);
  hipLaunchKernelGGL(route_any<kBF16>, dim3(nb), dim3(kAnyWaves * kWave), (size_t)(kAnyWaves + 1) * a.E * 4,
                     s, a);
  return nb;
}

template <bool kBF16, int LPT, int VPL, int WAVES>
void launch_back(const lrm_router& r, const void* logits, const int32_t* topk_idx,
                 const float* topk_w, const int32_t* counts, const float* adot, float* dlogits,
                 hipStream_t s) {
  constexpr int kTokens = WAVES * kWave / LPT;
  const unsigned nb = grid_for(((int64_t)r.T + kTokens - 1) / kTokens, 2048);
  const int vec = (int64_t)r.E * (kBF16 ? 2 : 4) % 16 == 0;
  hipLaunchKernelGGL((route_backward<kBF16, LPT, VPL, WAVES>), dim3(nb), dim3(WAVES * kWave),
                     (size_t)kTokens * r.E * 4, s, logits, topk_idx, topk_w, counts, adot, r.T, r.E,
                     r.k, r.gate, r.balance_coef, vec, dlogits);
}

template <bool kBF16>
void launch_back_e(const lrm_router& r, const void* logits, const int32_t* topk_idx,
                   const float* topk_w, const int32_t* counts, const float* adot, float* dlogits,
                   hipStream_t s) {
  // 32768 tokens: 19.2 us with 4 lanes a token; 1021: 6.6 with 4, 4.8 with 8, 4.2 with 16
  if (r.E <= 128 && r.T <= kShortBatch)
    return launch_back<kBF16, 16, 8, 4>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
  if (r.E <= 128) return launch_back<kBF16, 8, 16, 4>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
  if (r.E <= 256) return launch_back<kBF16, 8, 32, 4>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
  if (r.E <= 512) return launch_back<kBF16, 16, 32, 4>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
  launch_back<kBF16, 64, 64, 2>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
}

}  // namespace

hipError_t launch_route(const lrm_router& r, const void* logits, const uint8_t* mask,
                        int32_t* topk_idx, float* topk_w, float* lse, int32_t* counts, float* prob,
                        float* loss, char* ws, hipStream_t s) {
  const RouteWs wl = route_ws(r.E);
  const RouteArgs a{logits, mask, r.T, r.E, r.k, r.gate, topk_idx, topk_w, lse,
                    (int32_t*)(ws + wl.tokens), wl.pitch, (int32_t*)(ws + wl.counts),
                    (float*)(ws + wl.prob)};
  const RouteOut o{counts, prob, loss, (int32_t*)(ws + wl.err), r.balance_coef};
  const unsigned nb = r.dtype == LRM_BF16 ? launch_rows_any<true>(a, o, s) : launch_rows_any<false>(a, o, s);
  // route_rows of one workgroup ends with the results themselves: one launch for a short batch
  if (nb > 1 || r.k > 16)
    hipLaunchKernelGGL(route_final, dim3(1), dim3(kFinalThreads), 0, s, a.part_tokens, a.part_counts,
                       a.part_prob, (int)nb, r.E, wl.pitch, r.k, r.balance_coef, counts, prob, loss,
                       (int32_t*)(ws + wl.err));
  return hipGetLastError();
}

hipError_t launch_route_backward(const lrm_router& r, const void* logits, const int32_t* topk_idx,
                                 const float* topk_w, const int32_t* counts, const float* adot,
                                 float* dlogits, hipStream_t s) {
  if (r.dtype == LRM_BF16)
    launch_back_e<true>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
  else
    launch_back_e<false>(r, logits, topk_idx, topk_w, counts, adot, dlogits, s);
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
