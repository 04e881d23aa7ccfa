// lrm_grouped_fc1_swiglu, lrm_grouped_fc2, lrm_combine_tokens: the experts' forward products over
// the routed rows, and the return of their outputs to the tokens.
//
// For the rows r of local expert i (token t, pair p): [a; c] = W1_i x_t, phi_r = SiLU(a) c,
// y_r = W_i phi_r, out_t = residual_t + sum_p alpha_p y_r (LRMoE Appendix 7.1 Eq. (4): the layer
// whose backward the other calls compute).  Both products contract over the contiguous axis of
// both operands (rows of x or phi against rows of W1 or W).
//
// Products, activation and the sum over a token's rows are float32; ac, phi, y and out are rounded to
// the layer's type where they are stored.  ac and phi are what the backward takes in that type.  y in
// it halves the bytes of its way through memory, and adds sum_p |alpha_p| 2^-8 |y_p| to out's own error of
// 2^-8 |out|: more than that where a token's terms cancel.  A caller who does not want it gives float32
// rows (kWide).  Qwen3 share with the residual, bf16 / float32 rows: FC2 810-850 / 1030 us, combine 227 /
// 486, out against 64 bits 1.76e-3 / 1.66e-3 of its norm; one token: no difference in time.
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
// past the last one.  Every wave finds it by itself with a scan over 64 experts at a time, the
// offsets of 256 in flight, so no launch builds a table of tiles.
struct RowTile {
  int e, r0, r1;
};

template <int BM>
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ fwd_off, int E_loc, int cap,
                                             int64_t idx) {
  constexpr int B = 4;
  const int lane = lane_id();
  int64_t base = 0;
  for (int e0 = 0; e0 < E_loc; e0 += B * kWave) {
    int a[B], b[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = e0 + i * kWave + lane;
      a[i] = e < E_loc ? fwd_off[e] : 0;
      b[i] = e < E_loc ? fwd_off[e + 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (e0 + i * kWave >= E_loc) break;
      a[i] = clampi(a[i], 0, cap);
      b[i] = clampi(b[i], a[i], cap);
      const int n = (b[i] - a[i] + BM - 1) / BM;
      const int inc = wave_inclusive_scan(n);
      const uint64_t m = ballot(base + inc > idx);
      if (m) {
        const int l = __builtin_ctzll(m);
        const int r0 = __builtin_amdgcn_readlane(a[i] + (int)(idx - (base + inc - n)) * BM, l);
        const int end = __builtin_amdgcn_readlane(b[i], l);
        return {e0 + i * kWave + l, r0, r0 + BM < end ? r0 + BM : end};
      }
      base += __builtin_amdgcn_readlane(inc, kWave - 1);
    }
  }
  return {-1, 0, 0};
}

__device__ __forceinline__ float silu_mul(float a, float c) { return a / (1.0f + expf(-a)) * c; }

// The same with the hardware's power of two and reciprocal, for outputs that are rounded to bf16: the
// exact forms took 7 % of FC1's time.  Each is off by about 2^-23 of itself, the power by |a| 2^-23 more
// from its rounded argument (2^-16.5 at the largest a it tells from infinity, against the 2^-8 of bf16).
// exp(-a) = infinity gives 0, as it should.
__device__ __forceinline__ float silu_mul_fast(float a, float c) {
  return a * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f)) * c;
}

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
  int64_t units;   // the most units (row tile, column tile) there can be
};

// The token of pair p, or -1 for a pair id that is none.
__device__ __forceinline__ int64_t token_of(const FcArgs& g, int p) {
  return p >= 0 && p < g.P ? p / g.k : -1;
}

// Operands are read through buffer resources: a row or chunk that is not there gets an offset beyond
// the range and reads as zeros.
constexpr uint32_t kOutOfRange = 0x80000000u;

// The K step (of n) at which a unit of column block c of expert e starts; it takes the others in
// turn, cyclically.  Units that all start at 0 read the same few hundred bytes of every weight row at
// a time, and where the rows' pitch is a power of two those lie in a few of the memory's channels:
// FC1 of 32 tokens (h 2048, d 768, 150 MB of weights in use) took 45.0 us so and takes 37.5 (34.0 with
// the weights past the caches).  A row's sum depends on its expert and column alone among the rows of a
// problem; the tile shape, and with it the order, follows from the problem's sizes and capacity.
__device__ __forceinline__ int first_step(int c, int e, int n) {
  return (int)((5u * (unsigned)c + 7u * (unsigned)e) % (unsigned)n);
}

// Buffer resource of 2^31 bytes from base: every offset that is used lies below what the host checked.
// The base's words come from a vector instruction; a buffer access may read them five wait states
// later, which the compiler does not keep for the accesses in assembly statements (dma16).  The s_nop
// is that wait, and its outputs are what the loads read, so no vector instruction writes those again.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t operand(const char* base) {
  const uint64_t v = (uint64_t)(uintptr_t)base;
  uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  asm("s_nop 4" : "+s"(lo), "+s"(hi));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), (short)0,
                                           (int)kOutOfRange, 0x00020000);
}

// ------------------------------------------------------------------------------------------------
// float32 products: 64 rows x 128 weight rows (for kSwiglu 64 of each half, so 64 output columns) by 4
// wavefronts, each one 32 rows x two 32-wide column tiles, which for kSwiglu are the same columns of the
// gate and the up half.  Bound by the float32 matrix rate (64 cycles an MFMA, against three 16-byte LDS
// reads a lane for eight of them): the next K step's loads are in registers while one is multiplied, and
// a CU's many small workgroups cover each other's barriers.  A lane's 16 bytes hold four k of one row;
// the i-th MFMA takes the i-th of both operands, so k = 8 s + i and 8 s + 4 + i meet, in any order.
// kLong: runs of 128 k are summed apart and then added, so that a long row's sum is no less exact than
// a short one's; that second set of accumulators takes 124 registers a lane and leaves 4 workgroups a
// CU, without it 80 leave 6.
// ------------------------------------------------------------------------------------------------
constexpr int kBM = 64, kBNH = 64, kKS = 16, kPitch = kKS + 4, kRun = 128, kLongK = 512, kF32Threads = 256;

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

template <bool kSwiglu, bool kLong>
__global__ __launch_bounds__(kF32Threads, kLong ? 4 : 6) void fc_f32(FcArgs g) {
  constexpr int CH = kKS / 4;
  constexpr int NA = kBM * CH / kF32Threads, NB = 2 * kBNH * CH / kF32Threads;   // chunks a thread moves
  __shared__ __attribute__((aligned(16))) float sa[kBM * kPitch];
  __shared__ __attribute__((aligned(16))) float sb[2 * kBNH * kPitch];
  const int cols = (g.N + (kSwiglu ? kBNH : 2 * kBNH) - 1) / (kSwiglu ? kBNH : 2 * kBNH);
  const int tid = threadIdx.x, lane = lane_id(), wm = tid / kWave / 2, wn = tid / kWave % 2;
  const int kc = (tid % CH) * 4;   // this thread's k of a step
  for (int64_t u = blockIdx.x; u < g.units; u += gridDim.x) {   // unit = (row tile, column tile)
    const RowTile t = find_tile<kBM>(g.fwd_off, g.E_loc, g.cap, u / cols);
    if (t.e < 0) return;
    const int n0 = (int)(u % cols) * (kSwiglu ? kBNH : 2 * kBNH);
    const __amdgpu_buffer_rsrc_t ra = operand((const char*)g.A + (kSwiglu ? 0 : (int64_t)t.r0 * g.K * 4));
    const __amdgpu_buffer_rsrc_t rb =
        operand((const char*)g.B + (int64_t)t.e * (kSwiglu ? 2 : 1) * g.N * g.K * 4);
    uint32_t oa[NA], ob[NB];
#pragma unroll
    for (int j = 0; j < NA; ++j) {
      const int r = t.r0 + tid / CH + j * (kF32Threads / CH);
      int64_t src = -1;
      if (r < t.r1) {
        src = r - t.r0;
        if (kSwiglu) {
          src = token_of(g, g.row_pair[r]);
          if (src < 0) set_error(g.err, LRM_DEVERR_INDEX);
        }
      }
      oa[j] = src < 0 ? kOutOfRange : ((uint32_t)src * (uint32_t)g.K + kc) * 4;
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int r = tid / CH + j * (kF32Threads / CH);   // row of the B tile
      const int col = n0 + (kSwiglu ? r % kBNH : r);
      const uint32_t src = (uint32_t)(col + (kSwiglu ? r / kBNH * g.N : 0));
      ob[j] = col < g.N ? (src * (uint32_t)g.K + kc) * 4 : kOutOfRange;
    }
    uint4 va[NA], vb[NB];
    f32x16 acc[2], run[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] = run[j][i] = 0.0f;   // acc: only for kLong
#pragma unroll
    for (int j = 0; j < NA; ++j) va[j] = load16(ra, kc < g.K ? oa[j] : kOutOfRange);
#pragma unroll
    for (int j = 0; j < NB; ++j) vb[j] = load16(rb, kc < g.K ? ob[j] : kOutOfRange);
    for (int k0 = 0; k0 < g.K; k0 += kKS) {
      const int at = tid / CH * kPitch + kc;
#pragma unroll
      for (int j = 0; j < NA; ++j) *(uint4*)(sa + at + j * (kF32Threads / CH) * kPitch) = va[j];
#pragma unroll
      for (int j = 0; j < NB; ++j) *(uint4*)(sb + at + j * (kF32Threads / CH) * kPitch) = vb[j];
      __syncthreads();
      const bool in = k0 + kKS + kc < g.K;   // past the last step every load is out of range
#pragma unroll
      for (int j = 0; j < NA; ++j) va[j] = load16(ra, in ? oa[j] + (k0 + kKS) * 4 : kOutOfRange);
#pragma unroll
      for (int j = 0; j < NB; ++j) vb[j] = load16(rb, in ? ob[j] + (k0 + kKS) * 4 : kOutOfRange);
      __builtin_amdgcn_sched_barrier(0);   // a whole step ahead of their use
      const float* fa = sa + (wm * 32 + (lane & 31)) * kPitch + 4 * (lane >> 5);
      const float* fb = sb + (wn * 32 + (lane & 31)) * kPitch + 4 * (lane >> 5);
#pragma unroll
      for (int ks = 0; ks < kKS; ks += 8) {
        const float4 a = *(const float4*)(fa + ks);
        const float4 b0 = *(const float4*)(fb + ks), b1 = *(const float4*)(fb + kBNH * kPitch + ks);
        run[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x, b0.x, run[0], 0, 0, 0);
        run[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.x, b1.x, run[1], 0, 0, 0);
        run[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.y, b0.y, run[0], 0, 0, 0);
        run[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.y, b1.y, run[1], 0, 0, 0);
        run[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.z, b0.z, run[0], 0, 0, 0);
        run[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.z, b1.z, run[1], 0, 0, 0);
        run[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.w, b0.w, run[0], 0, 0, 0);
        run[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a.w, b1.w, run[1], 0, 0, 0);
      }
      if (kLong && ((k0 + kKS) % kRun == 0 || k0 + kKS >= g.K)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            acc[j][i] += run[j][i];
            run[j][i] = 0.0f;
          }
      }
      __syncthreads();
    }
    const f32x16(&sum)[2] = kLong ? acc : run;
    float* out = (float*)g.out;
    float* phi = (float*)g.out2;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t r = t.r0 + wm * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      const int col = n0 + wn * 32 + (lane & 31);
      if (r >= t.r1) continue;
      if constexpr (kSwiglu) {
        if (col >= g.N) continue;
        if (out != nullptr) {
          out[r * 2 * g.N + col] = sum[0][i];
          out[r * 2 * g.N + g.N + col] = sum[1][i];
        }
        phi[r * g.N + col] = silu_mul(sum[0][i], sum[1][i]);
      } else {
        if (col < g.N) out[r * g.N + col] = sum[0][i];
        if (col + kBNH < g.N) out[r * g.N + col + kBNH] = sum[1][i];
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// bf16 products of many rows an expert.
//
// A workgroup of WW x WT wavefronts computes BT tokens x BW weight rows; a wavefront owns MT x NT
// tiles of 32 x 32, the weights as the MFMA's row operand and the tokens as its columns, so a
// lane's accumulators hold consecutive outputs of one token.  For kSwiglu the weight rows of the
// tile are dealt in 32-row groups, gate, up, gate, up, .., so that both halves of an output column
// meet in one lane.  Both operands contract over their contiguous axis: K steps of 64 elements go
// from global memory straight to an LDS ring of S stages, the rows of x gathered by the load's
// per-lane offset.  One barrier a step, before its last slice: by then every wavefront holds that
// slice in registers, so the stage is free for the step S on, whose loads go out behind it.
// Workgroups are persistent; each die has a range of units of its own, whose panels share its L2.
//
// Bound by the matrix units at the clock that power leaves (1.6 GHz, 61 % busy), then by the loads:
// with every panel in L2 the GLM4.5 share's FC1 would be 8 % faster.  Measured: that FC1 (250k rows,
// h 4096, d 1408) 5.13-5.17 ms, 1120 TFLOP/s (a library product of 8192^3: 1314); FC2 of the Qwen3 share
// (250k rows, h 2048, d 768) 832 us, 945 TFLOP/s, a fifth of it outputs.  Tried and slower: four
// wavefronts of 128 x 128 (953), K steps of 32 in four stages (1054), waiting for the last unit's
// stores a step later (1091), staggered workgroups, blocks of 4 or 16 row tiles.
// ------------------------------------------------------------------------------------------------
constexpr int BK = 64;                                    // K step: rows of 128 bytes in LDS
constexpr int CH = 8;                                     // their 16-byte chunks

template <int WW_, int WT_, int MT_, int NT_, int S_, bool kSpread_ = false>
struct Shape {
  static constexpr int WW = WW_, WT = WT_, MT = MT_, NT = NT_, S = S_;
  static constexpr int NW = WW * WT, THREADS = NW * kWave;
  static constexpr int BW = 32 * MT * WW, BT = 32 * NT * WT;
  static constexpr int ROW = BK * 2;                      // bytes of a row in LDS
  static constexpr int SLICES = BK / 16;
  static constexpr int T_BYTES = BT * ROW, W_BYTES = BW * ROW, STG = T_BYTES + W_BYTES;
  static constexpr int IT = T_BYTES / 1024 / NW, IW = W_BYTES / 1024 / NW, I = IT + IW;
  static_assert(IT * 1024 * NW == T_BYTES && IW * 1024 * NW == W_BYTES, "whole 1 KiB blocks a wave");
  // For few rows an expert: units start at K steps of their own (see first_step), and the weights pass
  // the caches by: with one row tile an expert a workgroup reads every line of them alone.  A hot
  // expert's further row tiles read them from memory again, and a small layer's weights, which could
  // stay in the memory-side cache between calls, do not (two tokens, three sets of weights in turn:
  // 23.8 us against 19.5; twelve sets, as in a model: 22.9 against 24.8).
  static constexpr bool SPREAD = kSpread_;
  static constexpr int TABLE = 1024 + 1;                  // tiles before each expert
  // FC2's outputs go through 2 KiB of LDS a wavefront where as many workgroups still fit a CU.
  static constexpr int TABLE_BYTES = (TABLE + 3) / 4 * 16, OUT_BYTES = NW * 2048;
  static constexpr bool STAGED =
      160 * 1024 / (S * STG + TABLE_BYTES + OUT_BYTES) == 160 * 1024 / (S * STG + TABLE_BYTES);
  static constexpr int LDS = S * STG + TABLE_BYTES + (STAGED ? OUT_BYTES : 0);
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(S * I < 64, "vmcnt range");
};

// 16 bytes a lane from r + voff to LDS address lds + 16 lane.  Inline assembly, so that the compiler
// does not wait for it before every LDS read; the pipeline orders it with vmcnt and barriers.  The
// s_nop is the wait state that a load into LDS needs behind a write of M0: within a statement the
// compiler adds none.
template <bool kStream>
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff) {
  if constexpr (kStream)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(lds), "v"(voff), "s"(r)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(r)
                 : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ bf16x8 lds_b128(uint32_t addr) {
  return *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)addr;
}

// Chunk c of row r sits at chunk c ^ swizzle(r).  Two rows span the 64 banks, so any 16 rows that
// hold each value of (r / 2) % 8 twice, once in an even and once in an odd row, read 16 different
// 16-byte groups of banks at one k: so do the 16 lanes that a 16-byte LDS read serves at a time.
// (r % 8 instead would put rows r and r + 8 on the same banks: half of all LDS cycles were conflicts.)
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

// One output tile: token rows [r0, r1) of expert e, weight rows from n0.
struct Unit {
  int e, r0, r1, n0;
};

// Unit u of a die's range: tiles in blocks of kRowBlock row tiles, within a block rows fastest, so
// that the workgroups of a die share a few panels of both operands at a time.
constexpr int kRowBlock = 8;

template <class C, bool kSwiglu>
__device__ __forceinline__ Unit unit_of(const FcArgs& g, const int* before, int row_tiles, int cols,
                                        int64_t u) {
  const int64_t block = u / (kRowBlock * cols);
  const int within = (int)(u - block * kRowBlock * cols);
  const int left = row_tiles - (int)block * kRowBlock, rows = left < kRowBlock ? left : kRowBlock;
  const int tile = (int)block * kRowBlock + within % rows;
  int e = 0;
  for (int e0 = 0; e0 < g.E_loc; e0 += kWave) {   // the expert whose tiles hold `tile`
    const int lane = lane_id();
    const uint64_t m = ballot(e0 + lane < g.E_loc && before[e0 + lane + 1] > tile);
    if (m) {
      e = e0 + __builtin_ctzll(m);
      break;
    }
  }
  Unit t;
  t.e = __builtin_amdgcn_readfirstlane(e);
  const int a = clampi(g.fwd_off[t.e], 0, g.cap), b = clampi(g.fwd_off[t.e + 1], a, g.cap);
  t.r0 = a + (tile - before[t.e]) * C::BT;
  t.r1 = t.r0 + C::BT < b ? t.r0 + C::BT : b;
  t.n0 = within / rows * (kSwiglu ? C::BW / 2 : C::BW);
  return t;
}

// The loads, which run ahead of the products through the K steps of one unit and on into the next:
// a unit's epilogue and the next one's first loads then take place together.  Per lane: the source
// offset of each 16 bytes it moves, constant over a unit's K steps (the bases advance); lane l moves
// a chunk of row l / 8 of each 1 KiB block of 8 rows, chunk_of(q) in block q.
template <class C, bool kSwiglu>
struct Loader {
  uint32_t t[C::IT], w[C::IW];
  int pair[C::IT];       // the rows' pairs, fetched one step before the offsets are formed
  const char* pt;        // tokens and weights at k0
  const char* pw;
  int k0, wave, lane;
  int nk, left;          // K steps of a unit, and those still to load
  bool more;             // a unit is left to load

  // the chunk that belongs at position l % 8 of row 8 q + l / 8
  __device__ __forceinline__ int chunk_of(int q) const {
    return (lane % CH) ^ (lane / 16) ^ ((q & 1) << 2);
  }

  __device__ __forceinline__ void fetch(const FcArgs& g, const Unit& u) {
    if constexpr (kSwiglu) {
#pragma unroll
      for (int j = 0; j < C::IT; ++j) {
        const int r = u.r0 + (wave * C::IT + j) * CH + lane / CH;
        pair[j] = r < u.r1 ? g.row_pair[r] : 0;
      }
    }
  }

  __device__ __forceinline__ void begin(const FcArgs& g, const Unit& u) {
    const uint32_t pitch = (uint32_t)g.K * 2;
#pragma unroll
    for (int j = 0; j < C::IT; ++j) {
      const int r = u.r0 + (wave * C::IT + j) * CH + lane / CH;
      if constexpr (kSwiglu) {
        const bool ok = pair[j] >= 0 && pair[j] < g.P;
        if (!ok) set_error(g.err, LRM_DEVERR_INDEX);
        t[j] = r < u.r1 && ok ? (uint32_t)(pair[j] / g.k) * pitch + chunk_of(wave * C::IT + j) * 16
                              : kOutOfRange;
      } else {
        t[j] = r < u.r1 ? (uint32_t)(r - u.r0) * pitch + chunk_of(wave * C::IT + j) * 16 : kOutOfRange;
      }
    }
#pragma unroll
    for (int j = 0; j < C::IW; ++j) {
      const int row = (wave * C::IW + j) * CH + lane / CH;
      const int col = u.n0 + (kSwiglu ? row / 64 * 32 + row % 32 : row);
      const uint32_t src = kSwiglu && (row & 32) ? (uint32_t)(g.N + col) : (uint32_t)col;
      w[j] = col < g.N ? src * pitch + chunk_of(wave * C::IW + j) * 16 : kOutOfRange;
    }
    pt = (const char*)g.A + (kSwiglu ? 0 : (int64_t)u.r0 * g.K * 2);
    pw = (const char*)g.B + (int64_t)u.e * (kSwiglu ? 2 : 1) * g.N * g.K * 2;
    const int first = C::SPREAD ? first_step(u.n0 / (kSwiglu ? C::BW / 2 : C::BW), u.e, nk) : 0;
    k0 = first * BK;
    pt += first * C::ROW;
    pw += first * C::ROW;
    left = nk;
  }

  // Load q (tokens first) of the K step at k0 into the stage at LDS address `st`; where the step ends
  // past K, the chunks past it become zeros.
  template <int Q>
  __device__ __forceinline__ void load(uint32_t st, __amdgpu_buffer_rsrc_t rt, __amdgpu_buffer_rsrc_t rw,
                                       int K) const {
    const int q = Q < C::IT ? wave * C::IT + Q : wave * C::IW + Q - C::IT;
    uint32_t off;
    if constexpr (Q < C::IT) off = t[Q];
    else off = w[Q - C::IT];
    if (k0 + BK > K) off = k0 + chunk_of(q) * 8 < K ? off : kOutOfRange;
    dma16<(C::SPREAD && Q >= C::IT)>(Q < C::IT ? rt : rw, st + (Q < C::IT ? 0 : C::T_BYTES) + q * 1024, off);
  }
  template <int Q = 0>
  __device__ __forceinline__ void load_all(uint32_t st, __amdgpu_buffer_rsrc_t rt, __amdgpu_buffer_rsrc_t rw,
                                           int K) const {
    if constexpr (Q < C::I) {
      load<Q>(st, rt, rw, K);
      load_all<Q + 1>(st, rt, rw, K);
    }
  }
  __device__ __forceinline__ void step() {
    pt += C::ROW;
    pw += C::ROW;
    k0 += BK;
    --left;
    if (C::SPREAD && k0 >= nk * BK) {   // a spread unit's first steps come last
      k0 = 0;
      pt -= nk * C::ROW;
      pw -= nk * C::ROW;
    }
  }
};

template <class C>
struct Frags {
  bf16x8 w[C::MT], t[C::NT];
};

// Lane offsets (bytes from a stage) of this wavefront's fragments of each 16-wide slice.
template <class C>
struct Reads {
  uint32_t w[C::SLICES], t[C::SLICES];
};

template <class C>
__device__ __forceinline__ void read_frags(Frags<C>& f, const Reads<C>& r, uint32_t st, int slice) {
  const uint32_t pw = st + r.w[slice], pt = st + r.t[slice];
#pragma unroll
  for (int i = 0; i < C::MT; ++i) f.w[i] = lds_b128(pw + i * 32 * C::ROW);
#pragma unroll
  for (int j = 0; j < C::NT; ++j) f.t[j] = lds_b128(pt + j * 32 * C::ROW);
}

template <class C>
__device__ __forceinline__ void multiply(const Frags<C>& f, f32x16 (&acc)[C::MT][C::NT]) {
#pragma unroll
  for (int i = 0; i < C::MT; ++i)
#pragma unroll
    for (int j = 0; j < C::NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.w[i], f.t[j], acc[i][j], 0, 0, 0);
}

// Spreads the slice's LDS reads over its MFMAs.
template <class C>
__device__ __forceinline__ void interleave() {
  constexpr int M = C::MT * C::NT, R = (C::MT + C::NT + M - 1) / M;   // reads behind each MFMA
#pragma unroll
  for (int q = 0; q < M; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
  }
}

// 32 outputs of each of 32 tokens as bf16.  Accumulators hold columns 8 g + 4 (l / 32) + 0..3 of token
// l % 32 for g = 0..3; the halves of two groups change places between lanes l and l + 32, so that
// each lane has 8 consecutive columns: q[h] those from column 16 h + 8 (l / 32).
__device__ __forceinline__ void pack_tile(const float (&v)[16], uint4 (&q)[2]) {
  uint32_t p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto x = __builtin_amdgcn_permlane32_swap(p[4 * h], p[4 * h + 2], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(p[4 * h + 1], p[4 * h + 3], false, false);
    q[h] = make_uint4(x[0], y[0], x[1], y[1]);
  }
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// n packed 32-column tiles of 32 tokens from row r0 to out (rows of `pitch` elements, columns from
// `col`, those below `end` only, rows below r1 only), from where the lanes hold them: an instruction
// writes 32 rows by 32 bytes.
template <int n>
__device__ __forceinline__ void store_direct(const uint4 (&q)[n][2], uint16_t* out, int64_t pitch,
                                             int64_t r0, int64_t r1, int col, int end, int lane) {
  const int64_t r = r0 + (lane & 31);
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = col + 32 * i + 16 * h + 8 * (lane >> 5);
      if (r < r1 && c < end) *(uint4*)(out + r * pitch + c) = q[i][h];
    }
}

// Two unrounded 32-column tiles of 32 tokens to float32 rows, from where the lanes hold them.
__device__ __forceinline__ void store_wide(const f32x16& a, const f32x16& b, float* out, int64_t pitch,
                                           int64_t r0, int64_t r1, int col, int end, int lane) {
  const int64_t r = r0 + (lane & 31);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = col + 32 * i + 8 * q + 4 * (lane >> 5);
      const f32x16& v = i ? b : a;
      if (r < r1 && c < end)
        *(float4*)(out + r * pitch + c) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
}

// Two packed tiles (see store_direct) through `stage` (2 KiB of LDS, this wavefront's), 16 tokens at a time: an
// instruction writes 8 rows by 128 bytes.  FC2's outputs are 20 % of its time (a copy that stores
// nothing takes 673 us where the Qwen3 share takes 840 to 868); this saves 3 % of it.  FC1's, whose two
// halves and phi come in runs of 64 bytes a wavefront, were no faster this way.
__device__ __forceinline__ void store_staged(const uint4 (&q)[2][2], uint16_t* out, int64_t pitch,
                                             int64_t r0, int64_t r1, int col, int end, int lane,
                                             char* stage) {
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int tok = (lane & 31) - 16 * pass;
    if (tok >= 0 && tok < 16) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *(uint4*)(stage + tok * 128 + (((4 * i + 2 * h + (lane >> 5)) ^ tok) & 7) * 16) = q[i][h];
    }
    wave_fence();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = 8 * k + lane / 8, c = lane % 8;
      const uint4 v = *(const uint4*)(stage + t * 128 + ((c ^ t) & 7) * 16);
      const int64_t r = r0 + 16 * pass + t;
      if (r < r1 && col + 8 * c < end) *(uint4*)(out + r * pitch + col + 8 * c) = v;
    }
    wave_fence();
  }
}

template <class C, bool kSwiglu, bool kWide>
__global__ __launch_bounds__(C::THREADS) void fc_bf16(FcArgs g, int nxcd) {
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  int* before = (int*)(lds + C::S * C::STG);
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int ww = wave / C::WT, wt = wave % C::WT;
  // tiles before each expert
  if (wave == 0) {
    int base = 0;
    for (int e0 = 0; e0 < g.E_loc; e0 += kWave) {
      const int e = e0 + lane;
      int n = 0;
      if (e < g.E_loc) {
        const int a = clampi(g.fwd_off[e], 0, g.cap), b = clampi(g.fwd_off[e + 1], a, g.cap);
        n = (b - a + C::BT - 1) / C::BT;
      }
      const int inc = wave_inclusive_scan(n);
      if (e < g.E_loc) before[e + 1] = base + inc;
      base += __shfl(inc, kWave - 1, kWave);
    }
    if (lane == 0) before[0] = 0;
  }
  __syncthreads();
  const int row_tiles = __builtin_amdgcn_readfirstlane(before[g.E_loc]);
  const int bn = kSwiglu ? C::BW / 2 : C::BW, cols = (g.N + bn - 1) / bn;
  const int64_t total = (int64_t)row_tiles * cols, per = (total + nxcd - 1) / nxcd;
  const int64_t lo = (int64_t)(blockIdx.x % nxcd) * per, hi = lo + per < total ? lo + per : total;
  const int nb = gridDim.x / nxcd;

  const uint32_t ring = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)lds);
  Reads<C> rd;
#pragma unroll
  for (int s = 0; s < C::SLICES; ++s) {
    const uint32_t at = (lane & 31) * C::ROW + (((2 * s + (lane >> 5)) ^ swizzle(lane & 31)) << 4);
    rd.w[s] = C::T_BYTES + ww * C::MT * 32 * C::ROW + at;
    rd.t[s] = wt * C::NT * 32 * C::ROW + at;
  }
  int64_t u = lo + blockIdx.x / nxcd;
  if (u >= hi) return;
  Loader<C, kSwiglu> ld;
  ld.wave = wave;
  ld.lane = lane;
  const int nk = (g.K + BK - 1) / BK;
  ld.nk = nk;
  Unit t = unit_of<C, kSwiglu>(g, before, row_tiles, cols, u), nx = t;
  int64_t un = u;        // the loader's unit
  ld.fetch(g, t);
  ld.begin(g, t);
  ld.more = true;
  // the first S steps of the stream
  for (int s = 0; s < C::S; ++s) {
    if (ld.more) {
      ld.load_all(ring + s * C::STG, operand(ld.pt), operand(ld.pw), g.K);
      ld.step();
      if (ld.left == 0) {
        un += nb;
        ld.more = un < hi;
        if (ld.more) {
          nx = unit_of<C, kSwiglu>(g, before, row_tiles, cols, un);
          ld.fetch(g, nx);
          ld.begin(g, nx);
        }
      }
    }
  }
  wait_vm<0>();
  lds_barrier();
  uint32_t cur = ring;
  Frags<C> f[2];
  read_frags<C>(f[0], rd, cur, 0);
  for (; u < hi; u += nb) {
    f32x16 acc[C::MT][C::NT];
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int j = 0; j < C::NT; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
    for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
      for (int s = 0; s + 1 < C::SLICES; ++s) {
        read_frags<C>(f[(s + 1) & 1], rd, cur, s + 1);
        multiply<C>(f[s & 1], acc);
        interleave<C>();
        __builtin_amdgcn_sched_barrier(0);
      }
      // every fragment of this stage is in registers: once all waves are here it may be refilled;
      // the next stage has landed for every wave
      if (C::S > 2 && ld.more)
        wait_vm<(C::S - 2) * C::I>();
      else
        wait_vm<0>();
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's reads of the stage are done
      lds_barrier();
      const uint32_t next = cur + C::STG == ring + C::S * C::STG ? ring : cur + C::STG;
      if (ld.more && ld.left == 0) ld.begin(g, nx);
      __builtin_amdgcn_sched_barrier(0);
      if (ld.more) {
        const __amdgpu_buffer_rsrc_t rt = operand(ld.pt), rw = operand(ld.pw);
        ld.load_all(cur, rt, rw, g.K);
        ld.step();
        if (ld.left == 0) {   // the unit's last loads are out: its successor's rows
          un += nb;
          ld.more = un < hi;
          if (ld.more) {
            nx = unit_of<C, kSwiglu>(g, before, row_tiles, cols, un);
            ld.fetch(g, nx);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      read_frags<C>(f[C::SLICES & 1], rd, next, 0);
      multiply<C>(f[(C::SLICES - 1) & 1], acc);
      interleave<C>();
      __builtin_amdgcn_sched_barrier(0);
      cur = next;
    }
    static_assert(C::MT == 2, "a wavefront's columns: one gate and up pair, or two tiles");
#pragma unroll
    for (int j = 0; j < C::NT; ++j) {
      const int64_t r0 = t.r0 + (wt * C::NT + j) * 32;
      float v[16];
      if constexpr (kSwiglu) {
        const int col = t.n0 + ww * 32;
        uint4 q[1][2];
        if (g.out != nullptr) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = acc[i][j][k];
            pack_tile(v, q[0]);
            store_direct<1>(q, (uint16_t*)g.out + i * g.N, 2 * g.N, r0, t.r1, col, g.N, lane);
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = silu_mul_fast(acc[0][j][k], acc[1][j][k]);
        pack_tile(v, q[0]);
        store_direct<1>(q, (uint16_t*)g.out2, g.N, r0, t.r1, col, g.N, lane);
      } else if constexpr (kWide) {
        store_wide(acc[0][j], acc[1][j], (float*)g.out, g.N, r0, t.r1, t.n0 + ww * 64, g.N, lane);
      } else {
        uint4 q[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = acc[i][j][k];
          pack_tile(v, q[i]);
        }
        if constexpr (C::STAGED)
          store_staged(q, (uint16_t*)g.out, g.N, r0, t.r1, t.n0 + ww * 64, g.N, lane,
                       lds + C::S * C::STG + C::TABLE_BYTES + wave * 2048);
        else
          store_direct<2>(q, (uint16_t*)g.out, g.N, r0, t.r1, t.n0 + ww * 64, g.N, lane);
      }
    }
    // the loader is in the next unit, unless units are so short that it is past it already
    if (u + nb < hi) t = nk > C::S ? nx : unit_of<C, kSwiglu>(g, before, row_tiles, cols, u + nb);
  }
}

// ------------------------------------------------------------------------------------------------
// Few rows an expert (serving steps): bound by streaming the chosen experts' weights once.
//
// A workgroup computes up to 16 TT tokens x 32 weight rows (for kSwiglu 16 of each half) of one
// expert; its four wavefronts share the contracted axis, 128 bytes of every row in turn, so that
// even one token's eight experts put thousands of wavefronts' loads in flight at once.  Nothing
// goes through LDS but the four partial sums, added in a fixed order: a 16-row MFMA operand is one
// 16-byte load a lane (16 rows x 64 bytes), which for float32 serves four MFMAs, lane group q
// holding k = 4 q + i for the i-th (any order of k will do, as both operands have the same).
// Rows past the segment's end read its last row again and are not stored.  A tile holds the rows of
// any batch of up to 16 TT tokens (an expert is chosen once a token), so the weights are read
// once; the loads are temporal, as a row's 128-byte lines are read in two halves (non-temporal ones
// fetched them twice: 18 % slower).
// ------------------------------------------------------------------------------------------------
typedef float f32x4 __attribute__((ext_vector_type(4)));
constexpr int kFewWaves = 4;
constexpr int kFewAhead = 2;   // 128-byte pieces of each row in flight per wavefront
constexpr int WF = 2;          // 16-row weight operands

template <bool kBF16>
__device__ __forceinline__ f32x4 few_mma(uint4 a, uint4 b, f32x4 c) {
  if constexpr (kBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
}

// 128 bytes of 2 x 16 weight rows and TT x 16 token rows.
template <int TT>
struct FewPiece {
  uint4 a[2][WF], b[2][TT];
  __device__ __forceinline__ void load(const char* const (&pw)[WF], const char* const (&pt)[TT], int64_t off) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < WF; ++i) a[h][i] = *(const uint4*)(pw[i] + off + 64 * h);
#pragma unroll
      for (int j = 0; j < TT; ++j) b[h][j] = *(const uint4*)(pt[j] + off + 64 * h);
    }
  }
  // the last, partial piece: `left` elements from this lane's first, `half` of them 64 bytes on
  __device__ __forceinline__ void load_rest(const char* const (&pw)[WF], const char* const (&pt)[TT],
                                            int64_t off, int left, int half) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = left > h * half;
#pragma unroll
      for (int i = 0; i < WF; ++i) a[h][i] = in ? *(const uint4*)(pw[i] + off + 64 * h) : zero;
#pragma unroll
      for (int j = 0; j < TT; ++j) b[h][j] = in ? *(const uint4*)(pt[j] + off + 64 * h) : zero;
    }
  }
  template <bool kBF16>
  __device__ __forceinline__ void multiply(f32x4 (&acc)[WF][TT]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < WF; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[i][j] = few_mma<kBF16>(a[h][i], b[h][j], acc[i][j]);
  }
};

// One tile with TT token operands.
template <bool kBF16, bool kSwiglu, bool kWide, int TT>
__device__ __forceinline__ void few_tile(const FcArgs& g, const RowTile& t, int n0, int64_t u,
                                         f32x4 (*part)[kWave]) {
  constexpr int ESZ = kBF16 ? 2 : 4, V = 16 / ESZ;
  constexpr int STEP = 128 / ESZ;              // contracted elements of a 128-byte piece
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int64_t K = g.K;
  const int k0 = (lane >> 4) * V;              // this lane's elements of a 64-byte half piece
  const char* pt[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    int64_t r = t.r0 + 16 * j + (lane & 15);
    r = r < t.r1 ? r : t.r1 - 1;
    if (kSwiglu) r = token_of(g, g.row_pair[r]);
    pt[j] = (const char*)g.A + ((r < 0 ? 0 : r) * K + k0) * ESZ;   // a bad pair's outputs: below
  }
  const char* pw[WF];
#pragma unroll
  for (int i = 0; i < WF; ++i) {
    // columns past the last one read it again
    const int c = n0 + (kSwiglu ? 0 : 16 * i) + (lane & 15);
    const int64_t row = (c < g.N ? c : g.N - 1) + (kSwiglu && i ? (int64_t)g.N : 0);
    pw[i] = (const char*)g.B + ((int64_t)t.e * (kSwiglu ? 2 : 1) * g.N + row) * K * ESZ + k0 * ESZ;
  }
  f32x4 acc[WF][TT];
#pragma unroll
  for (int i = 0; i < WF; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // whole 128-byte pieces of the rows, this wavefront's w, w + 4, .. after a start that differs
  // between workgroups; then the row's rest
  const int whole = g.K / STEP;
  FewPiece<TT> f[kFewAhead];
  if (whole > 0) {
    const int first = first_step(n0 / (kSwiglu ? 16 : 32), t.e, whole);
    const auto piece = [&](int c) {
      const int at = (c < whole ? c : whole - 1) + first;
      return (int64_t)(at < whole ? at : at - whole) * 128;
    };
    // the loads run ahead without a condition, so that each wait is for one piece's loads alone;
    // past the end they fetch the last piece again
#pragma unroll
    for (int q = 0; q < kFewAhead; ++q) f[q].load(pw, pt, piece(w + q * kFewWaves));
    for (int c = w; c < whole; c += kFewAhead * kFewWaves) {
#pragma unroll
      for (int q = 0; q < kFewAhead; ++q) {
        if (c + q * kFewWaves < whole) f[q].template multiply<kBF16>(acc);
        f[q].load(pw, pt, piece(c + (kFewAhead + q) * kFewWaves));
      }
    }
  }
  if (g.K % STEP && whole % kFewWaves == w) {
    f[0].load_rest(pw, pt, (int64_t)whole * 128, g.K - whole * STEP - k0, STEP / 2);
    f[0].template multiply<kBF16>(acc);
  }
  // part[(wavefront, weight operand, token operand)]
#pragma unroll
  for (int i = 0; i < WF; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[(w * WF + i) * TT + j][lane] = acc[i][j];
  __syncthreads();
  // the wavefronts end the output operands in turn: lane l holds columns 4 (l / 16) + 0..3 of token
  // l % 16
  constexpr int OF = kSwiglu ? 1 : WF;
  for (int o = w; o < OF * TT; o += kFewWaves) {
    const int ci = o / TT, ti = o % TT;
    const int64_t r = t.r0 + 16 * ti + (lane & 15);
    f32x4 v = part[ci * TT + ti][lane], x = v;
#pragma unroll
    for (int q = 1; q < kFewWaves; ++q) v += part[(q * WF + ci) * TT + ti][lane];
    if constexpr (kSwiglu) {
      x = part[TT + ti][lane];
#pragma unroll
      for (int q = 1; q < kFewWaves; ++q) x += part[(q * WF + 1) * TT + ti][lane];
    }
    if (r < t.r1) {
      if (kSwiglu && token_of(g, g.row_pair[r]) < 0) {   // reads x as zeros
        v = x = (f32x4){0.f, 0.f, 0.f, 0.f};
        set_error(g.err, LRM_DEVERR_INDEX);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = n0 + 16 * ci + 4 * (lane >> 4) + i;
        if (c >= g.N) continue;
        if constexpr (kSwiglu) {
          if (g.out != nullptr) {
            store_elem<kBF16>(g.out, r * 2 * g.N + c, v[i]);
            store_elem<kBF16>(g.out, r * 2 * g.N + g.N + c, x[i]);
          }
          store_elem<kBF16>(g.out2, r * g.N + c, silu_mul(v[i], x[i]));
        } else {
          store_elem<kBF16 && !kWide>(g.out, r * g.N + c, v[i]);
        }
      }
    }
  }
  __syncthreads();
}

template <bool kBF16, bool kSwiglu, bool kWide, int TT>
__global__ __launch_bounds__(kFewWaves * kWave) void fc_few(FcArgs g) {
  constexpr int BN = kSwiglu ? 16 : 32;        // output columns
  __shared__ f32x4 part[kFewWaves * WF * TT][kWave];
  const int cols = (g.N + BN - 1) / BN;
  for (int64_t u = blockIdx.x; u < g.units; u += gridDim.x) {
    const RowTile t = find_tile<16 * TT>(g.fwd_off, g.E_loc, g.cap, u / cols);
    if (t.e < 0) return;
    const int n0 = (int)(u % cols) * BN, rows = t.r1 - t.r0;
    // as many token operands as the tile's rows need
    if (TT > 2 && rows > 32)
      few_tile<kBF16, kSwiglu, kWide, TT>(g, t, n0, u, part);
    else if (TT > 1 && rows > 16)
      few_tile<kBF16, kSwiglu, kWide, 2>(g, t, n0, u, part);
    else
      few_tile<kBF16, kSwiglu, kWide, 1>(g, t, n0, u, part);
  }
}

// Upper bound of the row tiles of bm rows: every expert's last may be partial, and none is empty.
inline int64_t most_tiles(const lrm_problem& p, int bm) {
  const int64_t most = (int64_t)p.L_cap / bm + p.E_loc;
  return most < p.L_cap ? most : p.L_cap;
}

inline unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 20) ? units : 1 << 20); }

template <bool kBF16, bool kSwiglu, bool kWide, int TT>
void launch_few(const lrm_problem& p, FcArgs g, hipStream_t s) {
  const int bn = kSwiglu ? 16 : 32;
  g.units = most_tiles(p, 16 * TT) * ((g.N + bn - 1) / bn);
  hipLaunchKernelGGL((fc_few<kBF16, kSwiglu, kWide, TT>), dim3(grid_of(g.units)), dim3(kFewWaves * kWave), 0, s, g);
}

// Workgroups of the persistent products: one a CU, a multiple of the dies.
constexpr int kDies = 8, kCUs = 256;

// The bf16 tiles, by tokens x weight rows.  Measured over a whole layer of 128 experts (h 2048, d 768,
// Zipf-skewed top-8 routing), us of FC1 / FC2 with Low, MidFew, Mid, Big:
//   256 tokens   61 / 35   67 / 39   83 / 40   78 / 55      (16 rows an expert on average)
//   512          96 / 51   81 / 43   90 / 43  124 / 55      (32)
//  1024         150 / 78  120 / 66  123 / 63  126 / 78      (64)
//  2048         271 / 142 168 / 105 164 / 103 185 / 104     (128)
//  4096         533 / 271 312 / 177 288 / 167 301 / 162     (256)
// and over a 16-expert share (h 4096, d 1408) at 256 tokens (64 rows) 148 / 72, 84 / 59, 101 / 62, 127 /
// 57, at 2048 922 / 437, 437 / 245, 425 / 238, 367 / 218.
using Low = Shape<2, 2, 2, 1, 3, true>;      // 64 x 128
using MidFew = Shape<4, 2, 2, 2, 3, true>;   // 128 x 256
using Mid = Shape<4, 2, 2, 2, 3>;
using Big = Shape<4, 2, 2, 4, 2>;            // 256 x 256
constexpr int kMidRows = 24, kSpreadRows = 96, kBigRows = 256;
// fc_few's share.  bf16: one token, while its experts make at most kFewUnits units of Low, half a unit a
// CU; us of FC1 / FC2 with fc_few against Low, of 8 experts in turn through 128:
//   h 1024, d 512    8.4 /  5.8 (64 and 64 units)    12.7 /  8.9
//   h 2048, d 768   17.4 /  9.1 (96, 128)            20.2 / 11.0
//   h 2048, d 1024  21.2 / 11.1 (128, 128)           20.4 / 12.7
//   h 4096, d 768   28.1 / 14.0 (96, 256)            34.8 / 12.9
//   h 4096, d 1024  30.8 / 18.7 (128, 256)           35.4 / 14.9
//   h 2560, d 1536  29.6 / 17.8 (192, 160)           27.4 / 17.3
//   h 4096, d 1408  39.9 / 21.8 (176, 256)           37.1 / 18.9
// and two tokens there 52.3 / 28.5 against 42.3 / 25.8.  float32 (h = d = 512, 32 experts) 27 / 19 against
// fc_f32's 44 / 32 at 64 tokens, 57 / 31 against 46 / 44 at 256.
constexpr int kFewBF16 = 1, kFewUnits = 128, kFewF32 = 128;

// The product has few enough rows and columns for fc_few; N its columns (of one half).
template <bool kBF16, bool kSwiglu>
bool takes_few(const lrm_problem& p, int N) {
  if (p.T > (kBF16 ? kFewBF16 : kFewF32)) return false;
  if (!kBF16) return true;
  const int bn = kSwiglu ? Low::BW / 2 : Low::BW;
  const int64_t local = (int64_t)p.T * p.k * p.E_loc / p.E;   // rows, and so experts, of a balanced load
  return (local > 1 ? local : 1) * ((N + bn - 1) / bn) <= kFewUnits;
}

template <class C, bool kSwiglu, bool kWide>
hipError_t launch_shape(const FcArgs& g, hipStream_t s) {
  constexpr int per_cu = 160 * 1024 / C::LDS;
  hipLaunchKernelGGL((fc_bf16<C, kSwiglu, kWide>), dim3(kCUs * per_cu), dim3(C::THREADS), 0, s, g, kDies);
  return hipGetLastError();
}

// kWide: a bf16 layer's y in float32.
template <bool kBF16, bool kSwiglu, bool kWide = false>
hipError_t launch_fc(const lrm_problem& p, FcArgs g, hipStream_t s) {
  if (p.L_cap == 0) return hipSuccess;   // no row
  if (takes_few<kBF16, kSwiglu>(p, g.N)) {   // an expert is chosen once a token: T rows at most
    if constexpr (kBF16) {
      launch_few<kBF16, kSwiglu, kWide, 1>(p, g, s);
    } else {
      if (p.T <= 16)
        launch_few<kBF16, kSwiglu, kWide, 1>(p, g, s);
      else if (p.T <= 32)
        launch_few<kBF16, kSwiglu, kWide, 2>(p, g, s);
      else
        launch_few<kBF16, kSwiglu, kWide, 4>(p, g, s);
    }
    return hipGetLastError();
  }
  if constexpr (kBF16) {
    // rows of an expert: the capacity's share, unless that is far above the balanced load T k / E (a
    // share of a layer has capacity for every pair).  Four times that load is for skewed routing; where a
    // share's is balanced, the shape is one for more rows than there are (the table: up to 13 % slower)
    const int64_t cap = (int64_t)p.L_cap / p.E_loc, most = 4 * ((int64_t)p.T * p.k / p.E);
    const int64_t rows = cap < most ? cap : most;
    if (rows >= kBigRows) return launch_shape<Big, kSwiglu, kWide>(g, s);
    if (rows >= kSpreadRows) return launch_shape<Mid, kSwiglu, kWide>(g, s);
    if (rows >= kMidRows) return launch_shape<MidFew, kSwiglu, kWide>(g, s);
    return launch_shape<Low, kSwiglu, kWide>(g, s);
  } else {
    const int bn = kSwiglu ? kBNH : 2 * kBNH;
    g.units = most_tiles(p, kBM) * ((g.N + bn - 1) / bn);
    if (g.K > kLongK)
      hipLaunchKernelGGL((fc_f32<kSwiglu, true>), dim3(grid_of(g.units)), dim3(kF32Threads), 0, s, g);
    else
      hipLaunchKernelGGL((fc_f32<kSwiglu, false>), dim3(grid_of(g.units)), dim3(kF32Threads), 0, s, g);
    return hipGetLastError();
  }
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

// The part of a row of y under one such chunk, in y's type: 16 bytes, or for a bf16 layer's float32 rows
// (kWide) 32.
template <bool kBF16, bool kWide>
struct RowPart {
  using C = Chunk<kBF16 && !kWide>;
  static constexpr int N = kWide ? 2 : 1;
  uint4 q[N];
  __device__ __forceinline__ void load(const uint4* row, int ch, bool in) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = in ? load_nt(row + ch * N + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void add(float w, float (&acc)[N * C::V]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[C::V];
      C::get(q[i], v);
#pragma unroll
      for (int j = 0; j < C::V; ++j) acc[i * C::V + j] += w * v[j];
    }
  }
};

// A wavefront sums kC 16-byte column chunks per lane of one token, in slot order in float32, the
// loads of B rows in flight together.  Memory-bound; with few tokens kC = 1 spreads a token's columns
// over wavefronts.  The token's rows come from the map (an entry counts only if it points inside
// [0, L) at a row that names the pair, so stale entries are ignored), or, with kScan (k <= 64), from a
// look through row_pair itself, which saves the launch that fills the map.  Every wavefront then reads
// all row ids, so that is for few of both; scan / map in us for 2048 columns in bf16:
//   256 rows,    32 tokens (128 wavefronts)  4.0 / 6.8     1024 rows, 128 tokens (512)    6.0 / 7.6
//   1024 rows,  512 tokens (2048)            5.5 / 5.8     1024 rows, 1024 tokens (4096)  6.7 / 5.7
//   1024 rows, 8192 tokens (32768)          31.8 / 13.3    1024 rows, 32768 tokens       89.4 / 26.5
constexpr int kScanRows = 1024, kScanWaves = 2048;

template <bool kBF16, bool kWide, bool kScan, int kC, int B>
__global__ __launch_bounds__(kBlock) void combine_tokens(const int32_t* __restrict__ map,
                                                         const int32_t* __restrict__ row_pair,
                                                         const int32_t* __restrict__ fwd_off,
                                                         int E_loc, int L_cap, int T, int k,
                                                         const float* __restrict__ topk_w,
                                                         const uint4* __restrict__ y, int hch,
                                                         const uint4* residual, uint4* out,
                                                         int32_t* __restrict__ err) {
  using C = Chunk<kBF16>;
  __shared__ int slots[kWavesPerBlock][kWave];
  const int lane = lane_id(), w = threadIdx.x / kWave;
  const int L = clampi(fwd_off[E_loc], 0, L_cap);
  const int parts = (hch + kC * kWave - 1) / (kC * kWave);
  const int64_t nw = (int64_t)gridDim.x * kWavesPerBlock;
  for (int64_t id = (int64_t)blockIdx.x * kWavesPerBlock + w; id < (int64_t)T * parts; id += nw) {
    const int64_t t = id / parts;
    const int c0 = (int)(id - t * parts) * kC * kWave + lane;
    float acc[kC][C::V];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int ch = c0 + c * kWave;
      if (residual != nullptr && ch < hch)
        C::get(load_nt(residual + t * hch + ch), acc[c]);
      else
        for (int q = 0; q < C::V; ++q) acc[c][q] = 0.0f;
    }
    if constexpr (kScan) {
      slots[w][lane] = -1;
      __builtin_amdgcn_wave_barrier();
      bool bad = false;
      for (int r = lane; r < L; r += kWave) {
        const int p = row_pair[r], j = p - (int)t * k;
        bad |= p < 0 || p >= (int64_t)T * k;
        if (j >= 0 && j < k) bad |= atomicExch(&slots[w][j], r) != -1;   // two rows of one pair
      }
      if (bad) set_error(err, LRM_DEVERR_INDEX);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    for (int j0 = 0; j0 < k; j0 += kWave) {
      const int64_t p = t * k + j0 + lane;
      int r = -1;
      float a = 0.0f;
      if (j0 + lane < k) {
        if constexpr (kScan) {
          r = slots[w][lane];
        } else {
          const int v = map[p];
          if (v >= 0 && v < L && row_pair[v] == p) r = v;
        }
        if (r >= 0) a = topk_w[p];
      }
      for (uint64_t m = ballot(r >= 0); m;) {   // slots in ascending order, B at a time
        RowPart<kBF16, kWide> x[B][kC];
        float wt[B];
        int n = 0;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (m == 0) break;
          const int jj = __builtin_ctzll(m);
          m &= m - 1;
          ++n;
          const uint4* src = y + (int64_t)__builtin_amdgcn_readlane(r, jj) * hch * (kWide ? 2 : 1);
          wt[b] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a), jj));
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int ch = c0 + c * kWave;
            x[b][c].load(src, ch, ch < hch);
          }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (b >= n) break;
#pragma unroll
          for (int c = 0; c < kC; ++c) x[b][c].add(wt[b], acc[c]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int ch = c0 + c * kWave;
      if (ch < hch) out[t * hch + ch] = C::put(acc[c]);
    }
  }
  if constexpr (!kScan) {
    // every row must own its map entry; two rows that name one pair leave one of them unread
    const int64_t n = (int64_t)gridDim.x * kBlock;
    for (int64_t r = (int64_t)blockIdx.x * kBlock + threadIdx.x; r < L; r += n) {
      const int p = row_pair[r];
      if (p >= 0 && p < (int64_t)T * k && map[p] != r) set_error(err, LRM_DEVERR_INDEX);
    }
  }
}

template <bool kBF16, bool kWide, bool kScan, int kC, int B>
void launch_tokens(const lrm_problem& p, const int32_t* map, const int32_t* row_pair,
                   const int32_t* fwd_off, const float* topk_w, const void* y, const void* residual,
                   void* out, int32_t* err, hipStream_t s) {
  const int hch = p.h * (kBF16 ? 2 : 4) / 16;
  const int64_t waves = (int64_t)p.T * ((hch + kC * kWave - 1) / (kC * kWave));
  const int64_t nb = (waves + kWavesPerBlock - 1) / kWavesPerBlock;
  hipLaunchKernelGGL((combine_tokens<kBF16, kWide, kScan, kC, B>), dim3((unsigned)(nb < 16384 ? nb : 16384)),
                     dim3(kBlock), 0, s, map, row_pair, fwd_off, p.E_loc, p.L_cap, p.T, p.k, topk_w,
                     (const uint4*)y, hch, (const uint4*)residual, (uint4*)out, err);
}

template <bool kBF16, bool kWide>
void launch_combine_t(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                      const float* topk_w, const void* y, const void* residual, void* out, char* ws,
                      hipStream_t s) {
  int32_t* err = (int32_t*)ws;
  int32_t* map = (int32_t*)(ws + kForwardMap);
  const int64_t waves = (int64_t)p.T * ((p.h * (kBF16 ? 2 : 4) / 16 + kWave - 1) / kWave);
  if (p.L_cap <= kScanRows && waves <= kScanWaves && p.k <= kWave) {
    launch_tokens<kBF16, kWide, true, 1, 8>(p, map, row_pair, fwd_off, topk_w, y, residual, out, err, s);
    return;
  }
  const int64_t lb = ((int64_t)p.L_cap + kBlock - 1) / kBlock;
  hipLaunchKernelGGL(forward_rows, dim3((unsigned)(lb < 1 ? 1 : (lb < 2048 ? lb : 2048))), dim3(kBlock), 0, s,
                     row_pair, fwd_off, p.E_loc, p.L_cap, (int64_t)p.T * p.k, map, err);
  launch_tokens<kBF16, kWide, false, 4, 2>(p, map, row_pair, fwd_off, topk_w, y, residual, out, err, s);
}

}  // namespace

hipError_t launch_fc1_swiglu(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                             const void* x, const void* W1, void* ac, void* phi, char* ws,
                             hipStream_t s) {
  const FcArgs g{x, W1, row_pair, fwd_off, (int64_t)p.T * p.k, p.E_loc, p.L_cap, p.k, p.h, p.d,
                 ac, phi, (int32_t*)ws, 0};
  return p.dtype == LRM_BF16 ? launch_fc<true, true>(p, g, s) : launch_fc<false, true>(p, g, s);
}

hipError_t launch_fc2(const lrm_problem& p, const int32_t* fwd_off, const void* phi, const void* W,
                      void* y, bool wide, hipStream_t s) {
  const FcArgs g{phi, W, nullptr, fwd_off, (int64_t)p.T * p.k, p.E_loc, p.L_cap, p.k, p.d, p.h,
                 y, nullptr, nullptr, 0};
  if (p.dtype != LRM_BF16) return launch_fc<false, false>(p, g, s);
  return wide ? launch_fc<true, false, true>(p, g, s) : launch_fc<true, false>(p, g, s);
}

hipError_t launch_combine(const lrm_problem& p, const int32_t* row_pair, const int32_t* fwd_off,
                          const float* topk_w, const void* y, bool wide, const void* residual, void* out,
                          char* ws, hipStream_t s) {
  if (p.dtype != LRM_BF16)
    launch_combine_t<false, false>(p, row_pair, fwd_off, topk_w, y, residual, out, ws, s);
  else if (wide)
    launch_combine_t<true, true>(p, row_pair, fwd_off, topk_w, y, residual, out, ws, s);
  else
    launch_combine_t<true, false>(p, row_pair, fwd_off, topk_w, y, residual, out, ws, s);
  return hipGetLastError();
}

}  // namespace lrm
