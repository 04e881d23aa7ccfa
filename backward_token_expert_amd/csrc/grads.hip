// lrm_grad_norm, lrm_clip_grads: the global norm of a list of tensors, and its clipping.
//
//   norm = sqrt(sum src^2),  dst = src * min(1, max_norm / norm)
// Squares of float32 and bf16 values are exact in float64, where they cannot overflow; the sums
// are float64 in a fixed order.  Bound by memory: src is read for the norm and again for the
// product, dst written once.
//
// The list is cut into chunks of kChunkBytes counted over all tensors, so that one launch's
// workgroups share many small tensors and one large one alike; a launch carries up to
// kTensorsPerLaunch entries in its kernel arguments (no copy of the list to the device, and a
// captured graph keeps its own).
#include <math.h>

#include "lrm_device.hpp"
#include "lrm_forward.hpp"

namespace lrm {
namespace {

constexpr int kBlock = 256;
constexpr int kInFlight = 8;                           // 16-byte accesses of a thread at a time
constexpr int64_t kKeepBytes = (int64_t)192 << 20;      // of a launch's end, for the second pass
constexpr int kChunkBytes = kBlock * kInFlight * 16;
__host__ __device__ constexpr int chunk_elems(bool bf16) { return kChunkBytes / (bf16 ? 2 : 4); }

struct GradList {
  int n;
  int64_t first[kTensorsPerLaunch + 1];  // first chunk of every entry; [n] = chunks in all
  const void* src[kTensorsPerLaunch];
  void* dst[kTensorsPerLaunch];
  int64_t count[kTensorsPerLaunch];
  uint8_t bf16[kTensorsPerLaunch];
};
static_assert(sizeof(GradList) < 4096, "kernel arguments");

// The entry that holds chunk c (uniform over the workgroup).
__device__ __forceinline__ int entry_of(const GradList& l, int64_t c) {
  int lo = 0, hi = l.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <bool kBF16>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if (kBF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

template <bool kBF16>
__device__ __forceinline__ double add_squares(double acc, uint4 q) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kBF16) {
      const double a = bf16_lo(w[j]), b = bf16_hi(w[j]);
      acc += a * a;
      acc += b * b;
    } else {
      const double a = __uint_as_float(w[j]);
      acc += a * a;
    }
  }
  return acc;
}

// Elements [i0, i1) of src, i0 a multiple of the chunk: this thread's sum of squares.  `keep`: the
// clipping reads them again soon; otherwise they pass the caches by.  (Up to kTensorsPerLaunch tensors
// the launch's end is the list's; of a longer list each launch keeps its own.)
template <bool kBF16>
__device__ __forceinline__ double chunk_squares(const void* src, int64_t i0, int64_t i1, bool keep) {
  constexpr int V = kBF16 ? 8 : 4;
  double acc = 0.0;
  if (((uintptr_t)src & 15) == 0) {
    const uint4* p = (const uint4*)src;
    if (i1 - i0 == chunk_elems(kBF16)) {
      uint4 q[kInFlight];
      const uint4* from = p + i0 / V + threadIdx.x;
      if (keep) {
#pragma unroll
        for (int j = 0; j < kInFlight; ++j) q[j] = from[j * kBlock];
      } else {
#pragma unroll
        for (int j = 0; j < kInFlight; ++j) q[j] = load_nt(from + j * kBlock);
      }
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) acc = add_squares<kBF16>(acc, q[j]);
      return acc;
    }
    const int64_t nv = i1 / V;
    for (int64_t v = i0 / V + threadIdx.x; v < nv; v += kBlock) acc = add_squares<kBF16>(acc, p[v]);
    i0 = nv * V > i0 ? nv * V : i0;
  }
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kBlock) {
    const double a = load_one<kBF16>(src, i);
    acc += a * a;
  }
  return acc;
}

// Sum over the workgroup's threads, in a fixed order; the result is thread 0's.
__device__ __forceinline__ double block_sum(double v, double* sh) {
  v = wave_sum(v);
  if (lane_id() == 0) sh[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < kBlock / kWave; ++w) s += sh[w];
  __syncthreads();
  return s;
}

__global__ __launch_bounds__(kBlock) void grad_squares(GradList l, double* __restrict__ part) {
  __shared__ double sh[kBlock / kWave];
  double acc = 0.0;
  for (int64_t c = blockIdx.x; c < l.first[l.n]; c += gridDim.x) {
    const int t = entry_of(l, c), n = chunk_elems(l.bf16[t]);
    const int64_t i0 = (c - l.first[t]) * n;
    const int64_t i1 = i0 + n < l.count[t] ? i0 + n : l.count[t];
    const bool keep = l.first[l.n] - c <= kKeepBytes / kChunkBytes;
    acc += l.bf16[t] ? chunk_squares<true>(l.src[t], i0, i1, keep)
                     : chunk_squares<false>(l.src[t], i0, i1, keep);
  }
  acc = block_sum(acc, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm from the partial sums of every launch, the same in every workgroup that calls it.
__device__ __forceinline__ float norm_of(const double* __restrict__ part, int64_t parts, double* sh) {
  double acc = 0.0;
  for (int64_t i = threadIdx.x; i < parts; i += kBlock) acc += part[i];
  return (float)sqrt(block_sum(acc, sh));
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

__global__ __launch_bounds__(kBlock) void grad_final(const double* __restrict__ part, int64_t parts,
                                                     float* __restrict__ norm,
                                                     int32_t* __restrict__ err) {
  __shared__ double sh[kBlock / kWave];
  const float n = norm_of(part, parts, sh);
  if (threadIdx.x == 0) {
    *norm = n;
    *err = finite(n) ? 0 : LRM_DEVERR_NONFINITE;
  }
}

template <bool kBF16>
__device__ __forceinline__ uint4 scaled(uint4 q, float f) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = kBF16 ? pack_bf16x2(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f)
                 : __float_as_uint(__uint_as_float(w[j]) * f);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void put16(uint4* p, uint4 v) {
  __builtin_nontemporal_store((u32x4){v.x, v.y, v.z, v.w}, (u32x4*)p);
}

template <bool kBF16>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, int64_t i0, int64_t i1,
                                            float f) {
  constexpr int V = kBF16 ? 8 : 4;
  if ((((uintptr_t)src | (uintptr_t)dst) & 15) == 0) {
    const uint4* p = (const uint4*)src;
    uint4* out = (uint4*)dst;
    if (i1 - i0 == chunk_elems(kBF16)) {
      uint4 q[kInFlight];
      const int64_t v = i0 / V + threadIdx.x;
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) q[j] = p[v + j * kBlock];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) put16(out + v + j * kBlock, scaled<kBF16>(q[j], f));
      return;
    }
    const int64_t nv = i1 / V;
    for (int64_t v = i0 / V + threadIdx.x; v < nv; v += kBlock) put16(out + v, scaled<kBF16>(p[v], f));
    i0 = nv * V > i0 ? nv * V : i0;
  }
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kBlock) {
    const float v = load_one<kBF16>(src, i) * f;
    if (kBF16)
      ((uint16_t*)dst)[i] = (uint16_t)pack_bf16x2(v, 0.0f);
    else
      ((float*)dst)[i] = v;
  }
}

// Every workgroup forms the norm from the partial sums itself, which saves a launch between the two
// passes: 8 KB from L2 for one launch of 1024 workgroups, as much again for every further one.  The
// chunks are taken from the last to the first: what the norm's pass read last is still in the
// memory-side cache (256 MB).
__global__ __launch_bounds__(kBlock) void grad_scale(GradList l, const double* __restrict__ part,
                                                     int64_t parts, float max_norm,
                                                     float* __restrict__ norm,
                                                     int32_t* __restrict__ err) {
  __shared__ double sh[kBlock / kWave];
  const float n = norm_of(part, parts, sh);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *norm = n;
    *err = finite(n) ? 0 : LRM_DEVERR_NONFINITE;
  }
  if (!finite(n)) return;
  const float f = n > max_norm ? max_norm / n : 1.0f;
  for (int64_t c = l.first[l.n] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = entry_of(l, c), m = chunk_elems(l.bf16[t]);
    if (f == 1.0f && l.src[t] == l.dst[t]) continue;   // in place, nothing to change
    const int64_t i0 = (c - l.first[t]) * m;
    const int64_t i1 = i0 + m < l.count[t] ? i0 + m : l.count[t];
    if (l.bf16[t])
      chunk_scale<true>(l.src[t], l.dst[t], i0, i1, f);
    else
      chunk_scale<false>(l.src[t], l.dst[t], i0, i1, f);
  }
}

// Entries [t0, t0 + kTensorsPerLaunch) of the list.
GradList slice(const lrm_tensor* list, int32_t n, int64_t t0) {
  GradList l;
  const int64_t left = n - t0;
  l.n = (int)(left < kTensorsPerLaunch ? (left < 0 ? 0 : left) : kTensorsPerLaunch);
  int64_t c = 0;
  for (int i = 0; i < l.n; ++i) {
    const lrm_tensor& t = list[t0 + i];
    l.first[i] = c;
    l.src[i] = t.src;
    l.dst[i] = t.dst;
    l.count[i] = t.count;
    l.bf16[i] = t.dtype == LRM_BF16;
    const int n = chunk_elems(l.bf16[i]);
    c += (t.count + n - 1) / n;
  }
  for (int i = l.n; i <= kTensorsPerLaunch; ++i) l.first[i] = c;
  return l;
}

int64_t launch_squares(const lrm_tensor* list, int32_t n, double* part, hipStream_t s) {
  int64_t parts = 0;
  for (int64_t q = 0; q < grad_launches(n); ++q) {
    const GradList l = slice(list, n, q * kTensorsPerLaunch);
    const int64_t c = l.first[l.n];
    const unsigned nb = (unsigned)(c < 1 ? 1 : (c < kGradBlocks ? c : kGradBlocks));
    hipLaunchKernelGGL(grad_squares, dim3(nb), dim3(kBlock), 0, s, l, part + parts);
    parts += nb;
  }
  return parts;
}

}  // namespace

hipError_t launch_grad_norm(const lrm_tensor* list, int32_t n, float* norm, char* ws,
                            hipStream_t s) {
  double* part = (double*)(ws + kGradPartials);
  const int64_t parts = launch_squares(list, n, part, s);
  hipLaunchKernelGGL(grad_final, dim3(1), dim3(kBlock), 0, s, part, parts, norm, (int32_t*)ws);
  return hipGetLastError();
}

hipError_t launch_clip(const lrm_tensor* list, int32_t n, float max_norm, float* norm, char* ws,
                       hipStream_t s) {
  double* part = (double*)(ws + kGradPartials);
  const int64_t parts = launch_squares(list, n, part, s);
  for (int64_t q = grad_launches(n) - 1; q >= 0; --q) {
    const GradList l = slice(list, n, q * kTensorsPerLaunch);
    const int64_t c = l.first[l.n];
    const unsigned nb = (unsigned)(c < 1 ? 1 : (c < kGradBlocks ? c : kGradBlocks));
    hipLaunchKernelGGL(grad_scale, dim3(nb), dim3(kBlock), 0, s, l, part, parts, max_norm, norm,
                       (int32_t*)ws);
  }
  return hipGetLastError();
}

}  // namespace lrm
