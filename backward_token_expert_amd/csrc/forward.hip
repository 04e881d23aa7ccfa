// lrm_grouped_fc1_swiglu, lrm_grouped_fc2, lrm_combine_tokens: the experts' forward products over
// the routed rows, and the return of their outputs to the tokens.
//
// For the rows r of local expert i (token t, pair p): [a; c] = W1_i x_t, phi_r = SiLU(a) c,
// y_r = W_i phi_r, out_t = residual_t + sum_p alpha_p y_r (LRMoE Appendix 7.1 Eq. (4): the layer
// whose backward the other calls compute).  Both products contract over the contiguous axis of
// both operands (rows of x or phi against rows of W1 or W).
#include <math.h>

#include "lrm_device.hpp"
#include "lrm_forward.hpp"

namespace lrm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBlock = 256;
constexpr int kWavesPerBlock = kBlock / kWave;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Row tile `idx` of the experts' segments cut into tiles of BM rows: expert and row range.  e = -1
// past the last one.  Every wave finds it by itself with one scan over 64 experts at a time, so no
// launch builds a table of tiles.
struct RowTile {
  int e, r0, r1;
};

template <int BM>
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ fwd_off, int E_loc, int cap,
                                             int idx) {
  const int lane = lane_id();
  int base = 0;
  for (int e0 = 0; e0 < E_loc; e0 += kWave) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < E_loc) {
      a = clampi(fwd_off[e], 0, cap);
      b = clampi(fwd_off[e + 1], a, cap);
    }
    const int n = (b - a + BM - 1) / BM;
    const int inc = wave_inclusive_scan(n);
    const uint64_t m = ballot(base + inc > idx);
    if (m) {
      const int l = __builtin_ctzll(m);
      const int r0 = __shfl(a + (idx - (base + inc - n)) * BM, l, kWave);
      const int end = __shfl(b, l, kWave);
      return {e0 + l, r0, r0 + BM < end ? r0 + BM : end};
    }
    base += __shfl(inc, kWave - 1, kWave);
  }
  return {-1, 0, 0};
}

__device__ __forceinline__ float silu_mul(float a, float c) { return a / (1.0f + expf(-a)) * c; }

template <bool kBF16>
__device__ __forceinline__ void store_elem(void* base, int64_t i, float v) {
  if (kBF16)
    ((uint16_t*)base)[i] = (uint16_t)pack_bf16x2(v, 0.0f);
  else
    ((float*)base)[i] = v;
}

// Arguments of one grouped product: rows of A (gathered through row_pair where it is set) against
// the rows of expert e's weights B + e * nb * K, K the contracted width.  kSwiglu: nb = 2d, out2 =
// phi, out = ac (or null).  Otherwise nb = h and out = y.
struct FcArgs {
  const void* A;
  const void* B;
  const int32_t* row_pair;
  const int32_t* fwd_off;
  int64_t P;
  int E_loc, cap, k, K, N;   // N: columns of one half (d), or of the product (h)
  void* out;
  void* out2;
  int32_t* err;
};

// 64 rows x 128 columns (for kSwiglu 64 of each half) by 4 wavefronts, each one 32 rows x two
// 32-wide column tiles, which for kSwiglu are the same columns of the gate and the up half.
constexpr int kBM = 64, kBNH = 64, kKS = 32;

template <bool kBF16, bool kSwiglu>
__global__ __launch_bounds__(kBlock) void fc_tile(FcArgs g) {
  constexpr int ESZ = kBF16 ? 2 : 4, V = 16 / ESZ, CH = kKS / V;  // elements, chunks per 16 bytes, row
  constexpr int PITCH = kBF16 ? kKS + 8 : kKS + 4;
  __shared__ __attribute__((aligned(16))) char sa[kBM * PITCH * ESZ];
  __shared__ __attribute__((aligned(16))) char sb[2 * kBNH * PITCH * ESZ];
  const int cols = (g.N + (kSwiglu ? kBNH : 2 * kBNH) - 1) / (kSwiglu ? kBNH : 2 * kBNH);
  for (int64_t u = blockIdx.x;; u += gridDim.x) {   // unit = (row tile, column tile)
  const RowTile t = find_tile<kBM>(g.fwd_off, g.E_loc, g.cap, (int)(u / cols));
  if (t.e < 0) return;
  const int n0 = (int)(u % cols) * (kSwiglu ? kBNH : 2 * kBNH);
  const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave, wm = w >> 1, wn = w & 1;
  const int64_t K = g.K;
  const char* We = (const char*)g.B + (int64_t)t.e * (kSwiglu ? 2 : 1) * g.N * K * ESZ;
  // this thread's chunks of A (one or two rows) and B
  constexpr int NA = kBM * CH / kBlock, NB = 2 * kBNH * CH / kBlock;
  const char* pa[NA];
  const char* pb[NB];
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int q = tid + j * kBlock, r = t.r0 + q / CH;
    int64_t src = -1;
    if (r < t.r1) {
      src = r;
      if (kSwiglu) {
        const int p = g.row_pair[r];
        src = p >= 0 && p < g.P ? p / g.k : -1;
        if (src < 0) set_error(g.err, LRM_DEVERR_INDEX);
      }
    }
    pa[j] = src < 0 ? nullptr : (const char*)g.A + (src * K + (q % CH) * V) * ESZ;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int q = tid + j * kBlock, r = q / CH;   // row of the B tile
    const int col = n0 + (kSwiglu ? r % kBNH : r);
    pb[j] = col < g.N ? We + ((int64_t)(col + (kSwiglu ? r / kBNH * g.N : 0)) * K + (q % CH) * V) * ESZ : nullptr;
  }
  f32x16 acc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.0f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = 0; k0 < g.K; k0 += kKS) {
#pragma unroll
    for (int j = 0; j < NA; ++j) {
      const int q = tid + j * kBlock, c = (q % CH) * V;
      *(uint4*)(sa + ((q / CH) * PITCH + c) * ESZ) =
          pa[j] && k0 + c < g.K ? *(const uint4*)(pa[j] + (int64_t)k0 * ESZ) : zero;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int q = tid + j * kBlock, c = (q % CH) * V;
      *(uint4*)(sb + ((q / CH) * PITCH + c) * ESZ) =
          pb[j] && k0 + c < g.K ? *(const uint4*)(pb[j] + (int64_t)k0 * ESZ) : zero;
    }
    __syncthreads();
    const int ra = wm * 32 + (lane & 31), rb = wn * 32 + (lane & 31);
    if constexpr (kBF16) {
#pragma unroll
      for (int ks = 0; ks < kKS; ks += 16) {
        const int c = ks + 8 * (lane >> 5);
        const bf16x8 a = *(const bf16x8*)(sa + (ra * PITCH + c) * 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bf16x8 b = *(const bf16x8*)(sb + ((rb + j * kBNH) * PITCH + c) * 2);
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[j], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < kKS; ks += 2) {
        const int c = ks + (lane >> 5);
        const float a = ((const float*)sa)[ra * PITCH + c];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(
              a, ((const float*)sb)[(rb + j * kBNH) * PITCH + c], acc[j], 0, 0, 0);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = t.r0 + wm * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
    if (r >= t.r1) continue;
    const int col = n0 + wn * 32 + (lane & 31);
    if (kSwiglu) {
      if (col < g.N) {
        if (g.out != nullptr) {
          store_elem<kBF16>(g.out, r * 2 * g.N + col, acc[0][i]);
          store_elem<kBF16>(g.out, r * 2 * g.N + g.N + col, acc[1][i]);
        }
        store_elem<kBF16>(g.out2, r * g.N + col, silu_mul(acc[0][i], acc[1][i]));
      }
    } else {
      if (col < g.N) store_elem<kBF16>(g.out, r * g.N + col, acc[0][i]);
      if (col + kBNH < g.N) store_elem<kBF16>(g.out, r * g.N + col + kBNH, acc[1][i]);
    }
  }
  }
}

template <bool kSwiglu>
hipError_t launch_fc(const lrm_problem& p, const FcArgs& g, hipStream_t s) {
  const int bn = kSwiglu ? kBNH : 2 * kBNH;
  // every expert's last tile may be partial
  const int64_t units = (((int64_t)p.L_cap + kBM - 1) / kBM + p.E_loc) * ((g.N + bn - 1) / bn);
  const dim3 grid((unsigned)(units < (1 << 20) ? units : 1 << 20));
  if (p.dtype == LRM_BF16)
    hipLaunchKernelGGL((fc_tile<true, kSwiglu>), grid, dim3(kBlock), 0, s, g);
  else
    hipLaunchKernelGGL((fc_tile<false, kSwiglu>), grid, dim3(kBlock), 0, s, g);
  return hipGetLastError();
}

// map[row_pair[r]] = r for every forward row; a pair id outside [0, P) sets LRM_DEVERR_INDEX.
__global__ __launch_bounds__(kBlock) void forward_rows(const int32_t* __restrict__ row_pair,
                                                       const int32_t* __restrict__ fwd_off,
                                                       int E_loc, int L_cap, int64_t P,
                                                       int32_t* __restrict__ map,
                                                       int32_t* __restrict__ err) {
  const int L = clampi(fwd_off[E_loc], 0, L_cap);
  for (int64_t r = (int64_t)blockIdx.x * kBlock + threadIdx.x; r < L; r += (int64_t)gridDim.x * kBlock) {
    const int p = row_pair[r];
    if (p >= 0 && p < P)
      map[p] = (int32_t)r;
    else
      set_error(err, LRM_DEVERR_INDEX);
  }
}

template <bool kBF16>
struct Chunk;  // 16 bytes as floats
template <>
struct Chunk<true> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void get(uint4 q, float (&v)[8]) {
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Chunk<false> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void get(uint4 q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

// One wavefront per token: the rows of its local pairs through the map (an entry counts only if it
// points inside [0, L) at a row that names the pair, so stale entries are ignored), summed in slot
// order in float32, kC 16-byte column chunks per lane at a time.  Memory-bound.
constexpr int kC = 4;

template <bool kBF16>
__global__ __launch_bounds__(kBlock) void combine_tokens(const int32_t* __restrict__ map,
                                                         const int32_t* __restrict__ row_pair,
                                                         const int32_t* __restrict__ fwd_off,
                                                         int E_loc, int L_cap, int T, int k,
                                                         const float* __restrict__ topk_w,
                                                         const uint4* __restrict__ y, int hch,
                                                         const uint4* residual, uint4* out,
                                                         int32_t* __restrict__ err) {
  using C = Chunk<kBF16>;
  const int lane = lane_id();
  const int L = clampi(fwd_off[E_loc], 0, L_cap);
  const int64_t nw = (int64_t)gridDim.x * kWavesPerBlock;
  for (int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; t < T; t += nw) {
    for (int c0 = 0; c0 < hch; c0 += kC * kWave) {
      float acc[kC][C::V];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int ch = c0 + lane + c * kWave;
        if (residual != nullptr && ch < hch)
          C::get(load_nt(residual + t * hch + ch), acc[c]);
        else
          for (int q = 0; q < C::V; ++q) acc[c][q] = 0.0f;
      }
      for (int j0 = 0; j0 < k; j0 += kWave) {
        const int64_t p = t * k + j0 + lane;
        int r = -1;
        float a = 0.0f;
        if (j0 + lane < k) {
          const int v = map[p];
          if (v >= 0 && v < L && row_pair[v] == p) {
            r = v;
            a = topk_w[p];
          }
        }
        for (uint64_t m = ballot(r >= 0); m; m &= m - 1) {   // slots in ascending order
          const int jj = __builtin_ctzll(m);
          const uint4* src = y + (int64_t)__shfl(r, jj, kWave) * hch;
          const float w = __shfl(a, jj, kWave);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int ch = c0 + lane + c * kWave;
            float v[C::V];
            C::get(ch < hch ? load_nt(src + ch) : make_uint4(0, 0, 0, 0), v);
#pragma unroll
            for (int q = 0; q < C::V; ++q) acc[c][q] += w * v[q];
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int ch = c0 + lane + c * kWave;
        if (ch < hch) out[t * hch + ch] = C::put(acc[c]);
      }
    }
  }
  // every row must own its map entry; two rows that name one pair leave one of them unread
  const int64_t n = (int64_t)gridDim.x * kBlock;
  for (int64_t r = (int64_t)blockIdx.x * kBlock + threadIdx.x; r < L; r += n) {
    const int p = row_pair[r];
    if (p >= 0 && p < (int64_t)T * k && map[p] != r) set_error(err, LRM_DEVERR_INDEX);
  }
}

}  // namespace

hipError_t launch_fc1_swiglu(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                             const void* x, const void* W1, void* ac, void* phi, char* ws,
                             hipStream_t s) {
  const FcArgs g{x, W1, row_pair, fwd_off, (int64_t)p.T * p.k, p.E_loc, p.L_cap, p.k, p.h, p.d,
                 ac, phi, (int32_t*)ws};
  return launch_fc<true>(p, g, s);
}

hipError_t launch_fc2(const lrm_problem& p, const int32_t* fwd_off, const void* phi, const void* W,
                      void* y, hipStream_t s) {
  const FcArgs g{phi, W, nullptr, fwd_off, (int64_t)p.T * p.k, p.E_loc, p.L_cap, p.k, p.d, p.h,
                 y, nullptr, nullptr};
  return launch_fc<false>(p, g, s);
}

hipError_t launch_combine(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                          const float* topk_w, const void* y, const void* residual, void* out,
                          char* ws, hipStream_t s) {
  int32_t* err = (int32_t*)ws;
  int32_t* map = (int32_t*)(ws + kForwardMap);
  const int64_t lb = ((int64_t)p.L_cap + kBlock - 1) / kBlock;
  hipLaunchKernelGGL(forward_rows, dim3((unsigned)(lb < 2048 ? lb : 2048)), dim3(kBlock), 0, s,
                     row_pair, fwd_off, p.E_loc, p.L_cap, (int64_t)p.T * p.k, map, err);
  const int64_t tb = ((int64_t)p.T + kWavesPerBlock - 1) / kWavesPerBlock;
  const unsigned nb = (unsigned)(tb < 16384 ? tb : 16384);
  const int hch = p.h * (p.dtype == LRM_BF16 ? 2 : 4) / 16;
  if (p.dtype == LRM_BF16)
    hipLaunchKernelGGL(combine_tokens<true>, dim3(nb), dim3(kBlock), 0, s, map, row_pair, fwd_off,
                       p.E_loc, p.L_cap, p.T, p.k, topk_w, (const uint4*)y, hch,
                       (const uint4*)residual, (uint4*)out, err);
  else
    hipLaunchKernelGGL(combine_tokens<false>, dim3(nb), dim3(kBlock), 0, s, map, row_pair, fwd_off,
                       p.E_loc, p.L_cap, p.T, p.k, topk_w, (const uint4*)y, hch,
                       (const uint4*)residual, (uint4*)out, err);
  return hipGetLastError();
}

}  // namespace lrm
