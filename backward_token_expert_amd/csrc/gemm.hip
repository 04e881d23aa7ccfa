// lrm_grouped_dw / lrm_grouped_dx: variable-size grouped FC2 gradients over the retained rows.
//
// LRMoE (arXiv 2610.37720) Sec. 3.2 Eq. (1) and Appendix 7.1 Eq. (8)-(9): the FC2 weight gradient
// of expert e is the sum of the retained pairs' rank-one contributions delta_u phi_u^T;
// Appendix 7.1 Eq. (4)-(7): the FC2 input gradient of a retained pair is W_e^T delta_u.
// Sec. 3.3/3.4 and Fig. 4: the retained count of an expert is the reduction dimension of the
// weight-gradient product and the row dimension of the input-gradient product, with no padding
// rows; counts and offsets (cmp_off) describe the segments.
//
//   dW[e]   (h x d) = Gc[seg e]^T (h x K_e) * Phic[seg e] (K_e x d)   reduction over rows
//   dphi    (K_e x d) = Gc[seg e] (K_e x h) * W[e] (h x d)            reduction over h
//
// bf16 (the production path): v_mfma_f32_32x32x16_bf16 with fp32 accumulation, workgroup tiles of
// 256 rows x 384 columns (8 wavefronts) or 256 x 256/192/128 (4 wavefronts), K step 32.  Operands
// are staged in LDS in their memory orientation by LDS-DMA and transposed on the LDS read (see the
// bf16 section).  The kernels are persistent: one workgroup per CU, and the work is laid out per
// XCD (the MI355X has 8 dies of 32 CUs, each with its own L2; workgroup ids are dealt to dies
// round-robin):
//   dW   the workgroups of a die form 1, 2 or 4 groups; experts are dealt to the groups (whole,
//        largest first, in a snake order, or, when that leaves a group far above the fair share,
//        cut along K into pieces whose later partial sums dw_fixup adds in piece order), and a
//        group walks the tiles of one job together, so every row of Gc/Phic is fetched from HBM
//        once per group and the other tiles of that job hit in L2;
//   dphi each die takes a contiguous range of (row tile, column tile) units (columns fastest, or
//        blocked for wide products, see dx_unit), so
//        a row tile's Gc rows and the expert's W stay in that die's L2; the one-launch kernel
//        (gemm_fused) runs its dW share first and then claims dphi units from these ranges.
// Global loads are issued S - 1 K steps ahead of their use through a ring of S LDS stages (S = 4
// for the 384-wide tile, 5 for the narrower ones).
// fp32: v_mfma_f32_32x32x2f32 on 64 x 64 tiles (four 32 x 32 wavefronts), plain grids.
// Expert sizes stay on the device: schedules are built by one-workgroup kernels from cmp_off; a
// zero-length segment writes zeros.  No atomics on the outputs (only on gemm_fused's unit
// counters): every output element is owned by one workgroup, so results are bitwise deterministic.
#include <mutex>
#include <type_traits>

#include "lrm_device.hpp"
#include "lrm_internal.hpp"

namespace lrm {

#ifdef LRM_TIMELINE
// Profiling builds only (build.py defines=("LRM_TIMELINE",), see timeline.py): per-workgroup
// timestamps of the one-launch GEMMs, from the 100 MHz clock: [0] start, [1] end of the dW share,
// [2] exit, [3] dphi units claimed, then (start, unit) of the first kTimelineUnits units; words
// 60 and 61 hold the shader-clock counter (s_memtime) at start and exit, the last two the hardware's
// XCC_ID (the die) and HW_ID (CU, SIMD and shader engine) registers.
constexpr int kTimelineWGs = 1024, kTimelineWords = 64, kTimelineUnits = 28;
static_assert(4 + 2 * kTimelineUnits <= kTimelineWords - 4, "unit stamps end before the last four words");
__device__ unsigned long long g_timeline[kTimelineWGs * kTimelineWords];
#endif

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kF32Threads = 256;  // fp32 path: 4 wavefronts in 2 x 2
constexpr int kBK = 32;           // bf16 K step
constexpr int kThreadsPerSchedule = 1024;

// ------------------------------------------------------------------------------------------------
// bf16 path
//
// Workgroup = 2 x WN wavefronts (2 along M, WN along N); a wavefront owns MT x NT tiles of 32 x 32,
// so the workgroup tile is (64 MT) x (32 NT WN).  Operands are staged in LDS in their memory
// orientation:
//   [k][mn] (mn contiguous): Gc and Phic for dW, W for dphi.  MFMA fragments are read with
//       ds_read_b64_tr_b16, which transposes 16-bit elements across each group of 16 lanes:
//       result lane i, element e = element (i % 4) of the 8 bytes that source lane 4e + i/4
//       addressed.  Source lane j therefore addresses row k0 + j/4, columns c0 + 4 (j % 4), and
//       result lane i receives column c0 + i at rows k0 .. k0+3; two such reads give the 8
//       consecutive reduction elements a 32x32x16 operand lane needs.
//   [mn][k] (k contiguous): Gc as the row operand of dphi; fragments are plain 16-byte reads.
// ------------------------------------------------------------------------------------------------
template <int MT_, int NT_, int WN_, bool AKMN_>
struct Tile {
  static constexpr int MT = MT_, NT = NT_, WN = WN_;
  static constexpr bool AKMN = AKMN_;
  static constexpr int NWAVES = 2 * WN, THREADS = NWAVES * kWave;
  static constexpr int BM = 64 * MT, BN = 32 * NT * WN;
  static constexpr int SA = BM * kBK;               // elements per LDS stage (no padding)
  static constexpr int SB = BN * kBK;
  static constexpr int IA = SA * 2 / 1024 / NWAVES;  // 1 KiB LDS-DMA loads per wavefront per stage
  static constexpr int IB = SB * 2 / 1024 / NWAVES;
  static_assert(IA * 1024 * NWAVES == SA * 2 && IB * 1024 * NWAVES == SB * 2, "tile / wavefronts");
  static_assert(BM % 128 == 0 && (BN % 128 == 0 || BN == 192), "swizzle needs these row widths");
};

// LDS layouts (element offsets).  Chunks of 8 elements (16 bytes) are XOR-swizzled inside a row
// instead of padding the pitch, because LDS-DMA writes 1 KiB contiguous blocks.
//   [k][mn], BMN wide: a 16-lane transpose read touches four consecutive rows, 32 bytes each, and
//     the next 16 lanes the next 32 bytes of the same rows.  With rows a multiple of 256 bytes all
//     rows start in the same bank, so chunk c of row r sits at chunk c ^ 4 (r % 4): the four rows
//     fall in four different 64-byte quarters of the 256-byte bank window.  With 384-byte rows
//     (BMN = 192) consecutive rows alternate between the two 128-byte halves, so chunk
//     c ^ 4 ((r / 2) % 2) separates rows r and r + 2 inside a half.
//   [mn][k], 32 wide: chunk c of row r sits at chunk c ^ ((r / 4) % 4), so 16 consecutive rows
//     read at one k offset hit 16 different 16-byte bank groups.
template <int BMN>
__device__ __forceinline__ int swz_chunk(int row) {
  return BMN == 192 ? ((row >> 1) & 1) << 2 : (row & 3) << 2;
}
template <int BMN>
__device__ __forceinline__ int swz_kmn(int row, int col) {
  return row * BMN + ((((col >> 3) ^ swz_chunk<BMN>(row))) << 3) + (col & 7);
}
__device__ __forceinline__ int swz_mnk(int row, int k) {
  return row * kBK + ((((k >> 3) ^ ((row >> 2) & 3))) << 3) + (k & 7);
}

// Global loads go straight to LDS (buffer_load_dwordx4 ... lds: lane l's 16 bytes land at the
// wave-uniform LDS address in M0 + 16 l).  Buffer resources end at the last valid row, so rows
// past a segment read as zeros in hardware; chunks past the matrix edge get an offset beyond any
// range.
constexpr uint32_t kOutOfRange = 0x80000000u;

constexpr int64_t kMaxWindow = 0x7FFFFFF0;

// Buffer resource over [base, base + bytes), bytes in [0, kMaxWindow], both uniform over the wave.
// Its words come from vector instructions; a buffer access may read them five wait states later, which
// the compiler does not keep for the accesses in assembly statements (dma16).  The s_nop is that wait,
// and its outputs are what the loads read, so no vector instruction writes those again.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const char* base, int bytes) {
  const uint64_t v = (uint64_t)(uintptr_t)base;
  uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  bytes = __builtin_amdgcn_readfirstlane(bytes);
  asm("s_nop 4" : "+s"(lo), "+s"(hi), "+s"(bytes));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), (short)0,
                                           bytes, 0x00020000);
}

// The load is written as inline assembly: the compiler then does not track it as an LDS write
// and does not drain all outstanding loads before every LDS read; the pipeline below orders the
// stages with explicit vmcnt waits and barriers instead.  M0 = lds + OFF (LDS byte address).  The
// sum is formed outside the assembly: an s_add inside it would overwrite SCC, which the compiler
// may hold live across the statement.  The s_nop is the wait state that a load into LDS needs behind
// a write of M0: within a statement the compiler adds none.
template <int OFF>
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds + OFF), "v"(voff), "s"(r)
               : "memory", "m0");
}

typedef __attribute__((address_space(3))) uint16_t lds_u16;

__device__ __forceinline__ uint32_t lds_addr(const uint16_t* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_u16*)p);
}

template <int OFF>
__device__ __forceinline__ s16x4 ds_tr16_at(uint32_t addr) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(uintptr_t)(addr + OFF));
}

template <int OFF>
__device__ __forceinline__ bf16x8 ds_b128_at(uint32_t addr) {
  return *(const __attribute__((address_space(3))) bf16x8*)(uintptr_t)(addr + OFF);
}

// LDS ring of S stages; stage s holds the A tile (SA elements) then the B tile (SB elements).
template <class C, int S>
struct Ring {
  static constexpr int A_BYTES = C::SA * 2, B_BYTES = C::SB * 2;
  static constexpr int STG = A_BYTES + B_BYTES, BYTES = S * STG;
  static_assert(BYTES <= 160 * 1024, "LDS ring exceeds 160 KiB");
};

// LDS stages: as many as fit in 160 KiB, at most 5.
template <class C>
constexpr int stages_for() {
  return (160 * 1024) / ((C::SA + C::SB) * 2) < 5 ? (160 * 1024) / ((C::SA + C::SB) * 2) : 5;
}

// Columns are dealt to the wavefronts interleaved: column sub-tile j of wavefront column wn starts
// at 32 wn + 32 WN j, so a tile whose last columns lie past the matrix edge leaves every
// wavefront the same number of live sub-tiles (a prefix j < NTA), and the wavefronts skip the
// MFMAs and fragment reads of the dead ones together instead of one SIMD idling the others.
template <class C>
__device__ __forceinline__ int col_of(int wn, int j) {
  return 32 * wn + 32 * C::WN * j;
}

// Live column sub-tiles of wavefront column wn when `ncols` columns of the tile are inside the
// matrix.
template <class C>
__device__ __forceinline__ int live_cols(int wn, int ncols) {
  const int r = ncols - 32 * wn;
  const int n = r <= 0 ? 0 : (r + 32 * C::WN - 1) / (32 * C::WN);
  return n > C::NT ? C::NT : n;
}

// Lane-dependent byte offsets (within a stage) of this wavefront's fragment reads, fixed for the
// whole kernel.  [k][mn] operands: offset of the first of the two transpose reads at k = 0; the
// second read is 4 rows on and the k = 16 slice 16 rows on, both constants.  [mn][k] operand:
// one offset per 16-wide slice (the chunk swizzle differs between them).
template <class C>
struct FragOffsets {
  uint32_t a[C::MT][C::AKMN ? 1 : 2];
  uint32_t b[C::NT];
};

template <int BMN>
__device__ __forceinline__ uint32_t kmn_offset(int base, int lane) {
  const int row = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int col = base + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  return (uint32_t)swz_kmn<BMN>(row, col) * 2;
}

template <class C>
__device__ __forceinline__ FragOffsets<C> frag_offsets(int wm, int wn, int lane) {
  FragOffsets<C> f;
#pragma unroll
  for (int i = 0; i < C::MT; ++i) {
    const int base = wm * 32 * C::MT + i * 32;
    if constexpr (C::AKMN) {
      f.a[i][0] = kmn_offset<C::BM>(base, lane);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f.a[i][h] = (uint32_t)swz_mnk(base + (lane & 31), 16 * h + 8 * (lane >> 5)) * 2;
    }
  }
#pragma unroll
  for (int j = 0; j < C::NT; ++j)
    f.b[j] = C::SA * 2 + kmn_offset<C::BN>(col_of<C>(wn, j), lane);
  return f;
}

// Single fragments of 16-wide slice H (0: k 0..15, 1: k 16..31) of the stage at LDS byte
// address `st`.
template <class C, int H>
__device__ __forceinline__ bf16x8 read_a(uint32_t st, const FragOffsets<C>& f, int i) {
  if constexpr (C::AKMN) {
    const uint32_t p = st + f.a[i][0];
    const s16x4 lo = ds_tr16_at<H * 16 * C::BM * 2>(p);
    const s16x4 hi = ds_tr16_at<(H * 16 + 4) * C::BM * 2>(p);
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    return ds_b128_at<0>(st + f.a[i][H]);
  }
}

template <class C, int H>
__device__ __forceinline__ bf16x8 read_b(uint32_t st, const FragOffsets<C>& f, int j) {
  const uint32_t p = st + f.b[j];
  const s16x4 lo = ds_tr16_at<H * 16 * C::BN * 2>(p);
  const s16x4 hi = ds_tr16_at<(H * 16 + 4) * C::BN * 2>(p);
  return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// One half step, row-streamed: the MFMAs of the current slice (B fragments bc and the first A
// fragment a0c already in registers), reading the current slice's later A rows just ahead of their
// use and the next slice's fragments (bn, a0n) along the way, so at most 2 NT + 2 fragments are
// live.  Scheduling groups alternate one MFMA with LDS reads, so the reads hide behind the matrix
// work.  `hook` runs once, after the MFMAs of the first A row have been issued (the second half
// step issues the ring's next loads there, behind matrix work instead of in front of it); a
// wavefront without live column sub-tiles (NT = 0) only runs the hook.
struct NoHook {
  __device__ __forceinline__ void operator()() const {}
};

template <class C, int HC, int HN, int NT, class Hook>
__device__ __forceinline__ void half_step(uint32_t sc, uint32_t sn, const FragOffsets<C>& fo,
                                          const bf16x8 (&bc)[C::NT], const bf16x8& a0c,
                                          bf16x8 (&bn)[C::NT], bf16x8& a0n,
                                          f32x16 (&acc)[C::MT][C::NT], const Hook& hook) {
  // NT (<= C::NT): the live column sub-tiles; the dead ones are neither read nor multiplied
  constexpr int MT = C::MT;
  constexpr int kReadA = C::AKMN ? 2 : 1;   // LDS read instructions per A fragment
  constexpr int kReads = kReadA * MT + 2 * NT;  // LDS read instructions per slice
  constexpr bool kHook = !std::is_same<Hook, NoHook>::value;
  if constexpr (NT > 0) {
    bf16x8 a = a0c;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      bf16x8 an;
      if (i + 1 < MT) an = read_a<C, HC>(sc, fo, i + 1);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j * MT / NT == i) bn[j] = read_b<C, HN>(sn, fo, j);
      if (i == MT - 1) a0n = read_a<C, HN>(sn, fo, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, bc[j], acc[i][j], 0, 0, 0);
      if (i + 1 < MT) a = an;
      if (kHook && i == 0) {
        // LDS reads issued with row 0: A row 1 and the B fragments dealt to row 0
        constexpr int r0 = (MT > 1 ? kReadA : 0) + 2 * ((NT + MT - 1) / MT);
        constexpr int per0 = (r0 + NT - 1) / NT;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, per0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        hook();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (kHook && MT > 1) {
      constexpr int r1 = kReads - ((MT > 1 ? kReadA : 0) + 2 * ((NT + MT - 1) / MT));
      constexpr int kMfma = (MT - 1) * NT;
      constexpr int per = (r1 + kMfma - 1) / kMfma;
#pragma unroll
      for (int q = 0; q < kMfma; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
      }
    } else if constexpr (!kHook) {
      constexpr int kMfma = MT * NT;
      constexpr int per = (kReads + kMfma - 1) / kMfma;
#pragma unroll
      for (int q = 0; q < kMfma; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
      }
    }
  } else {
    hook();
  }
}

// Per-lane source offsets (bytes, relative to the stage's first row / the tile's first row) of the
// DMA loads this wavefront issues for one stage.
template <int BMN, int I>
__device__ __forceinline__ void dma_offs_kmn(int64_t ld, int mn0, int mnend, int w, int lane,
                                             uint32_t (&o)[I]) {
#pragma unroll
  for (int j = 0; j < I; ++j) {
    const int q = (w * I + j) * 64 + lane, row = q / (BMN / 8);
    const int c = (q % (BMN / 8)) ^ swz_chunk<BMN>(row);
    const int col = mn0 + 8 * c;
    o[j] = col < mnend ? (uint32_t)((row * ld + col) * 2) : kOutOfRange;
  }
}

template <int I>
__device__ __forceinline__ void dma_offs_mnk(int64_t ld, int w, int lane, uint32_t (&o)[I],
                                             int (&kc)[I]) {
#pragma unroll
  for (int j = 0; j < I; ++j) {
    const int q = (w * I + j) * 64 + lane, row = q / 4;
    const int c = (q % 4) ^ ((row >> 2) & 3);
    kc[j] = 8 * c;
    o[j] = (uint32_t)((row * ld + 8 * c) * 2);
  }
}

// Operands of one output tile.  A: [k][mn] (AKMN) or [mn][k]; B: always [k][mn].
struct Operands {
  const uint16_t* A;
  int64_t lda;
  int a_mn0, a_mnend;
  const uint16_t* B;
  int64_t ldb;
  int b_mn0, b_mnend;
  int kbeg, kend;
};

// Barrier for LDS reuse: the waves have already waited for their own loads (vmcnt); no memory
// fence (which would wait for every outstanding load) is wanted here.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// s_waitcnt vmcnt(n) with the other counters left alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

template <int V>
struct IntC {
  static constexpr int value = V;
};

// Calls f(IntC<0>{}) .. f(IntC<N-1>{}) (compile-time indices, e.g. for instruction immediates).
template <int N, int J = 0, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (J < N) {
    f(IntC<J>{});
    static_for<N, J + 1>(f);
  }
}

// Issues the DMA loads of one K step.  kmn operands move their buffer window down the K rows; the
// [mn][k] operand moves its window along the rows and masks the chunks past kend when the step is
// partial.  Past the end of the K range every load falls outside its window and writes zeros.
// prepare() forms the next step's buffer resources (scalar work only), fire() issues its loads,
// advance() moves to the step after; the mainloop places the scalar work where matrix work hides
// it.
template <class C>
struct Loader {
  uint32_t oa[C::IA], ob[C::IB];
  int kca[C::IA];
  const char* pa;  // window bases of the next step
  const char* pb;
  int64_t sa, sb;  // bytes the bases move per step
  int rowa, rowb;  // [k][mn] operands: bytes per K row
  int ra;          // [mn][k] A: bytes from pa to the end of the tile's last row (<= kMaxWindow)
  int k0, kend;
  int na, nb;      // window bytes of the next step (prepare())

  __device__ __forceinline__ void init(const Operands& o, int w, int lane) {
    if constexpr (C::AKMN) {
      dma_offs_kmn<C::BM, C::IA>(o.lda, o.a_mn0, o.a_mnend, w, lane, oa);
      pa = (const char*)(o.A + (int64_t)o.kbeg * o.lda);
      rowa = (int)(o.lda * 2);
      sa = (int64_t)kBK * o.lda * 2;
    } else {
      dma_offs_mnk<C::IA>(o.lda, w, lane, oa, kca);
      pa = (const char*)(o.A + (int64_t)o.a_mn0 * o.lda + o.kbeg);
      const int64_t r = (int64_t)(o.a_mnend - o.a_mn0) * o.lda * 2 - (int64_t)o.kbeg * 2;
      ra = (int)(r <= 0 ? 0 : (r > kMaxWindow ? kMaxWindow : r));
      sa = kBK * 2;
    }
    dma_offs_kmn<C::BN, C::IB>(o.ldb, o.b_mn0, o.b_mnend, w, lane, ob);
    pb = (const char*)(o.B + (int64_t)o.kbeg * o.ldb);
    rowb = (int)(o.ldb * 2);
    sb = (int64_t)kBK * o.ldb * 2;
    k0 = o.kbeg;
    kend = o.kend;
  }

  __device__ __forceinline__ void prepare() {
    int rows = kend - k0;
    rows = rows < 0 ? 0 : (rows > kBK ? kBK : rows);
    na = C::AKMN ? rows * rowa : ra;
    nb = rows * rowb;
  }

  // wa / wb: LDS byte addresses of this wave's first 1 KiB block of the A / B part of the stage.
  __device__ __forceinline__ void fire(uint32_t wa, uint32_t wb) const {
    const __amdgpu_buffer_rsrc_t r_a = make_rsrc(pa, na);
    const __amdgpu_buffer_rsrc_t r_b = make_rsrc(pb, nb);
    if (C::AKMN || k0 + kBK <= kend) {
      static_for<C::IA>([&](auto j) { dma16<decltype(j)::value * 1024>(r_a, wa, oa[decltype(j)::value]); });
    } else {
      static_for<C::IA>([&](auto j) {
        constexpr int J = decltype(j)::value;
        dma16<J * 1024>(r_a, wa, k0 + kca[J] < kend ? oa[J] : kOutOfRange);
      });
    }
    static_for<C::IB>([&](auto j) { dma16<decltype(j)::value * 1024>(r_b, wb, ob[decltype(j)::value]); });
  }

  __device__ __forceinline__ void advance() {
    pa += sa;
    pb += sb;
    if constexpr (!C::AKMN) ra = ra > kBK * 2 ? ra - kBK * 2 : 0;
    k0 += kBK;
  }
};

// acc += A^T-or-A * B over k in [kbeg, kend), in K steps of 32 through the S-stage LDS ring at
// LDS byte address `ring`.
//
// Step kt runs in two halves.  First half: the MFMAs of slice 0 (fragments already in registers)
// while this wave reads slice 1 of the same stage.  Middle: wait for this wave's loads of stage
// kt+1, barrier (stage kt+1 is then complete in LDS for every wave, and every wave is done with
// stage kt-1), and issue the loads of step kt+S-1 into stage kt-1.  Second half: the MFMAs of
// slice 1 while reading slice 0 of stage kt+1.  Loads are issued for every step, past the end of
// the K range too (they fall outside their windows and write zeros), so the number of loads in
// flight at each wait is the same constant.  Ends with every load drained and a barrier, so the
// ring may be reused right away.
template <class C, int S, int NTA>
__device__ __forceinline__ void mainloop(const Operands& o, uint32_t ring, const FragOffsets<C>& fo,
                                         int w, int lane, f32x16 (&acc)[C::MT][C::NT]) {
  using R = Ring<C, S>;
  constexpr int I = C::IA + C::IB;
  static_assert(S >= 3 && (S - 2) * I < 64, "vmcnt range");
  const int nk = o.kend > o.kbeg ? (o.kend - o.kbeg + kBK - 1) / kBK : 0;
  if (nk == 0) return;
  Loader<C> ld;
  ld.init(o, w, lane);
  // this wave's first DMA block inside a stage, for the A and the B part
  const uint32_t blk_a = w * C::IA * 1024, blk_b = R::A_BYTES + w * C::IB * 1024;
#pragma unroll
  for (int st = 0; st < S - 1; ++st) {
    ld.prepare();
    ld.fire(ring + st * R::STG + blk_a, ring + st * R::STG + blk_b);
    ld.advance();
  }
  ld.prepare();
  wait_vm<(S - 2) * I>();
  lds_barrier();
  uint32_t rd = ring;                        // stage kt
  uint32_t wr = ring + (S - 1) * R::STG;     // stage kt - 1 (the DMA target)
  bf16x8 bA[C::NT], bB[C::NT], aA, aB;
  if constexpr (NTA > 0) {
    aA = read_a<C, 0>(rd, fo, 0);
#pragma unroll
    for (int j = 0; j < NTA; ++j) bA[j] = read_b<C, 0>(rd, fo, j);
  }
  for (int kt = 0; kt < nk; ++kt) {
    // first half: slice 0 of stage kt; reads slice 1 of the same stage
    half_step<C, 0, 1, NTA>(rd, rd, fo, bA, aA, bB, aB, acc, NoHook{});
    __builtin_amdgcn_sched_barrier(0);
    // middle: stage kt+1 complete for every wave; stage kt-1 free
    wait_vm<(S - 3) * I>();
    lds_barrier();
    const uint32_t rn = rd + R::STG == ring + R::BYTES ? ring : rd + R::STG;
    __builtin_amdgcn_sched_barrier(0);
    // second half: slice 1 of stage kt; reads slice 0 of stage kt+1 (unused after the last
    // step); the loads of step kt+S-1 into stage kt-1 go out after its first A row's MFMAs
    const uint32_t wa = wr + blk_a, wb = wr + blk_b;
    half_step<C, 1, 0, NTA>(rd, rn, fo, bB, aB, bA, aA, acc, [&] { ld.fire(wa, wb); });
    __builtin_amdgcn_sched_barrier(0);
    ld.advance();
    ld.prepare();
    wr = wr + R::STG == ring + R::BYTES ? ring : wr + R::STG;
    rd = rn;
  }
  wait_vm<0>();
  lds_barrier();
}

// The mainloop specialised for the wavefront's live column sub-tiles `nta` (wave-uniform).  Every
// specialisation issues the same loads and barriers, so the wavefronts of one workgroup may take
// different ones.
template <class C, int S, int NTA = C::NT>
__device__ __forceinline__ void mainloop_live(int nta, const Operands& o, uint32_t ring,
                                              const FragOffsets<C>& fo, int w, int lane,
                                              f32x16 (&acc)[C::MT][C::NT]) {
  if constexpr (NTA == 0) {
    mainloop<C, S, 0>(o, ring, fo, w, lane, acc);
  } else {
    if (nta >= NTA)
      mainloop<C, S, NTA>(o, ring, fo, w, lane, acc);
    else
      mainloop_live<C, S, NTA - 1>(nta, o, ring, fo, w, lane, acc);
  }
}

template <int MT, int NT>
__device__ __forceinline__ void zero_acc(f32x16 (&acc)[MT][NT]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
}

// C[m][n] for the wavefront's MT x NT tiles (columns dealt as col_of), rows < mend and columns
// < nend only.
// 32x32 accumulator layout: lane l holds column l % 32, rows 8 (r / 4) + 4 (l / 32) + r % 4.
// The stores are non-temporal: the float32 outputs are not read again by the launch, and keeping
// them out of L2 leaves it to the operand panels the other workgroups still reuse.
template <int MT, int NT, int WN>
__device__ __forceinline__ void store_acc(float* __restrict__ out, int64_t ldo, int m0, int mend,
                                          int n0, int nend, int wm, int wn, int lane,
                                          const f32x16 (&acc)[MT][NT]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = n0 + 32 * wn + 32 * WN * j + (lane & 31);   // interleaved, as col_of
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = m0 + wm * 32 * MT + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (m < mend && n < nend)
          __builtin_nontemporal_store(acc[i][j][r], out + (int64_t)m * ldo + n);
      }
    }
}

// dW: persistent.  The workgroups of a die form gpx groups of gs = nb / gpx; group g has a list of
// jobs (expert, K range, output) built by dw_schedule, and its workgroups take the units
// u = j, j + gs, ... of that list (unit = job-major, tile-minor), so they sweep one job's tiles
// together and its rows come from HBM once per group.  A job's tiles are ordered in column strips
// of kDwStrip column tiles, row by row within a strip: the gs tiles in flight then cover a block of
// about gs / kDwStrip row tiles by kDwStrip column tiles, whose operand panels a die's L2 holds,
// instead of a few whole rows of tiles when the product is wide.  A job whose output is a slot
// writes a partial sum of a split expert there (dw_fixup adds it); otherwise it writes dW
// directly.
constexpr int kDwStrip = 4;

// This workgroup's share of the dW units: group `grp`'s job list, and units j, j + gs, ...
struct DwPlan {
  const int32_t* jobs;
  int tn, tm, tpe, units, j, gs;
};

template <class C>
__device__ __forceinline__ DwPlan dw_plan(const int32_t* __restrict__ sched, int nxcd, int E_loc,
                                          int h, int d) {
  DwPlan p;
  p.tn = (d + C::BN - 1) / C::BN;
  p.tm = (h + C::BM - 1) / C::BM;
  p.tpe = p.tm * p.tn;
  const int x = blockIdx.x % nxcd, i = blockIdx.x / nxcd, nb = gridDim.x / nxcd;
  const int gpx = sched[1];
  p.gs = nb / gpx;
  const int grp = x * gpx + i / p.gs;
  p.j = i % p.gs;
  p.units = sched[4 + 3 * kMaxDwSlots + grp] * p.tpe;
  p.jobs = sched + kDwHeader + (int64_t)grp * dw_jobs_per_group(E_loc) * 4;
  return p;
}

// Unit u (job u / tpe, tile u % tpe) of a group's job list `jobs` (nothing for a skip record).
template <class C, int S>
__device__ __forceinline__ void dw_unit(const int32_t* __restrict__ jobs, int tm, int tn, int u,
                                       const uint16_t* __restrict__ Gc,
                                       const uint16_t* __restrict__ Phic, int E_loc, int K_cap,
                                       int h, int d, float* __restrict__ dW,
                                       float* __restrict__ slots, uint32_t ring_addr,
                                       f32x16 (&acc)[C::MT][C::NT]) {
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wm = w / C::WN, wn = w % C::WN;
  const FragOffsets<C> fo = frag_offsets<C>(wm, wn, lane);
  const int tpe = tm * tn;
  const int32_t* jb = jobs + 4 * (u / tpe);
  const int e = jb[0], kb = jb[1], ke = jb[2], slot = jb[3], local = u % tpe;
  if (slot == -2) return;  // an empty piece of a split expert
  // a record outside the buffers (never written so by dw_schedule) is skipped, not followed
  if (e < 0 || e >= E_loc || kb < 0 || ke < kb || ke > K_cap || slot < -1 || slot >= kMaxDwSlots)
    return;
  const int strip = local / (tm * kDwStrip), within = local - strip * tm * kDwStrip;
  const int sw = tn - strip * kDwStrip < kDwStrip ? tn - strip * kDwStrip : kDwStrip;
  const int m0 = (within / sw) * C::BM, n0 = (strip * kDwStrip + within % sw) * C::BN;
  const Operands o{Gc, h, m0, h, Phic, d, n0, d, kb, ke};
  zero_acc(acc);
  mainloop_live<C, S>(live_cols<C>(wn, d - n0), o, ring_addr, fo, w, lane, acc);
  float* out = slot < 0 ? dW + (int64_t)e * h * d : slots + (int64_t)slot * h * d;
  store_acc<C::MT, C::NT, C::WN>(out, d, m0, h, n0, d, wm, wn, lane, acc);
}

template <class C, int S>
__global__ __launch_bounds__(C::THREADS) void dw_bf16(const uint16_t* __restrict__ Gc,
                                                     const uint16_t* __restrict__ Phic,
                                                     const int32_t* __restrict__ sched, int nxcd,
                                                     int E_loc, int K_cap, int h, int d,
                                                     float* __restrict__ dW,
                                                     float* __restrict__ slots) {
  using R = Ring<C, S>;
  __shared__ __attribute__((aligned(1024))) uint16_t ring[R::BYTES / 2];
  const DwPlan pl = dw_plan<C>(sched, nxcd, E_loc, h, d);
  f32x16 acc[C::MT][C::NT];
  for (int u = pl.j; u < pl.units; u += pl.gs)
    dw_unit<C, S>(pl.jobs, pl.tm, pl.tn, u, Gc, Phic, E_loc, K_cap, h, d, dW, slots,
                  lds_addr(ring), acc);
}

// dW of each split expert += its partial slots, in piece order.  A fixed grid of kFixupBlocks
// workgroups strides over the split experts' elements (the expert loop is uniform), so the launch
// is small when nothing is split -- the usual case -- and still spreads a split expert's h x d
// elements over the whole chip.
constexpr int kFixupBlocks = 1024;

// Thread t of n adds the split experts' partial slots to dW (h * d a multiple of 4).
__device__ __forceinline__ void fixup_split_experts(const int32_t* __restrict__ sched, int E_loc,
                                                    int h, int d, const float* __restrict__ slots,
                                                    float* __restrict__ dW, int64_t t, int64_t n) {
  const int nsplit = sched[2];
  const int64_t n4 = (int64_t)h * d / 4;
  for (int sp = 0; sp < nsplit && sp < kMaxDwSlots; ++sp) {
    const int e = sched[4 + 3 * sp], first = sched[5 + 3 * sp], extra = sched[6 + 3 * sp];
    if (e < 0 || e >= E_loc || first < 0 || extra < 0 || first + extra > kMaxDwSlots) continue;
    float4* out = (float4*)(dW + (int64_t)e * h * d);
    for (int64_t q = t; q < n4; q += n) {
      float4 v = out[q];
      for (int k = 0; k < extra; ++k) {
        const float4 a = ((const float4*)(slots + (int64_t)(first + k) * h * d))[q];
        v.x += a.x;
        v.y += a.y;
        v.z += a.z;
        v.w += a.w;
      }
      out[q] = v;
    }
  }
}

__global__ __launch_bounds__(256) void dw_fixup(const int32_t* __restrict__ sched, int E_loc,
                                                int h, int d,
                                                const float* __restrict__ slots,
                                                float* __restrict__ dW) {
  fixup_split_experts(sched, E_loc, h, d, slots, dW, (int64_t)blockIdx.x * 256 + threadIdx.x,
                      (int64_t)kFixupBlocks * 256);
}

constexpr int kDxBlockRows = 8;

// dphi units = (row tile from the tile table, column tile), blocked: unit u covers rows
// [m0, min(m0 + BM, end of its expert's segment)) and columns [n0, n0 + BN).
template <class C, int S>
__device__ __forceinline__ void dx_unit(const uint16_t* __restrict__ Gc,
                                        const uint16_t* __restrict__ W,
                                        const int32_t* __restrict__ cmp_off,
                                        const int32_t* __restrict__ tiles, int u, int K_cap, int h,
                                        int d, float* __restrict__ dphi, uint32_t ring_addr,
                                        f32x16 (&acc)[C::MT][C::NT]) {
  const int tn = (d + C::BN - 1) / C::BN;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wm = w / C::WN, wn = w % C::WN;
  const FragOffsets<C> fo = frag_offsets<C>(wm, wn, lane);
  // Wide products (4 column tiles or more) take their units in blocks of kDxBlockRows row
  // tiles -- within a block rows fastest, then columns -- so that the units in flight on a die
  // span a few column panels of W and a block's row panels instead of every panel of W; narrower
  // ones take columns fastest (blocks of one row).  The last block may have fewer rows.
  const int rows = tiles[0];
  const int R = tn >= 4 ? kDxBlockRows : 1;
  const int blk = u / (R * tn), within = u - blk * R * tn;
  const int rb = rows - blk * R < R ? rows - blk * R : R;
  const int mt = blk * R + within % rb, n0 = (within / rb) * C::BN;
  const int e = tiles[1 + 2 * mt], m0 = tiles[2 + 2 * mt];
  int mend = cmp_off[e + 1];
  mend = mend > K_cap ? K_cap : mend;
  const Operands o{Gc, h, m0, mend, W + (int64_t)e * h * d, d, n0, d, 0, h};
  zero_acc(acc);
  mainloop_live<C, S>(live_cols<C>(wn, d - n0), o, ring_addr, fo, w, lane, acc);
  store_acc<C::MT, C::NT, C::WN>(dphi, d, m0, mend, n0, d, wm, wn, lane, acc);
}

// dphi: persistent, die x owns the contiguous unit range [x * per, (x + 1) * per).
template <class C, int S>
__global__ __launch_bounds__(C::THREADS) void dx_bf16(const uint16_t* __restrict__ Gc,
                                                     const uint16_t* __restrict__ W,
                                                     const int32_t* __restrict__ cmp_off,
                                                     const int32_t* __restrict__ tiles, int nxcd,
                                                     int K_cap, int h, int d,
                                                     float* __restrict__ dphi) {
  using R = Ring<C, S>;
  __shared__ __attribute__((aligned(1024))) uint16_t ring[R::BYTES / 2];
  const int tn = (d + C::BN - 1) / C::BN;
  const int total = tiles[0] * tn, per = (total + nxcd - 1) / nxcd;
  const int x = blockIdx.x % nxcd, i = blockIdx.x / nxcd, nb = gridDim.x / nxcd;
  const int u0 = x * per, u1 = u0 + per < total ? u0 + per : total;
  f32x16 acc[C::MT][C::NT];
  for (int u = u0 + i; u < u1; u += nb)
    dx_unit<C, S>(Gc, W, cmp_off, tiles, u, K_cap, h, d, dphi, lds_addr(ring), acc);
}

// Arguments of the one-launch GEMMs.
struct FusedArgs {
  const uint16_t* Gc;
  const uint16_t* Phic;
  const uint16_t* W;
  const int32_t* cmp_off;
  const int32_t* sched;
  const int32_t* tiles;
  int32_t* queue;
  int nxcd, E_loc, K_cap, h, d;
  float* dW;
  float* slots;
  float* dphi;
};

// The work loop of gemm_fused.  MIX (dw_schedule sets the flag): every workgroup starts with a
// dphi unit, then alternates dW and dphi units, and takes its dW units from one counter over all
// groups' lists instead of its group's fixed share.  Flag 1, store-bound products (dW jobs that
// average fewer K steps than a job's fixed cost, such as a whole layer with many empty experts):
// the dphi units, whose reads would wait behind the flood of dW tile stores, start first and the
// stores fill in around them on whichever workgroups are free; the counter walks the groups'
// lists one after the other.  Flag 2, one round of dphi units that would otherwise run after the
// dW shares and set the end of the launch (a few experts holding most rows): the counter walks
// the experts largest first, so the free workgroups start the longest dW jobs at once.
// Otherwise a workgroup runs its group's dW units first, in step with the group (for L2 reuse),
// then claims dphi units.
template <class CW, class CX, int S, bool MIX>
__device__ __forceinline__ void fused_loop(const FusedArgs& a, volatile int* claimed,
                                           uint32_t ring_addr, f32x16 (&acc)[CX::MT][CX::NT],
                                           unsigned long long* stamp) {
#ifdef LRM_TIMELINE
  int claims = 0;
#else
  (void)stamp;
#endif
  const DwPlan pl = dw_plan<CW>(a.sched, a.nxcd, a.E_loc, a.h, a.d);
  const int tn = (a.d + CX::BN - 1) / CX::BN;
  const int total = a.tiles[0] * tn, per = (total + a.nxcd - 1) / a.nxcd;
  const int x = blockIdx.x % a.nxcd;
  if constexpr (!MIX) {
    // the group's dW units, then dphi claims until every range is exhausted
    for (int u = pl.j; u < pl.units; u += pl.gs)
      dw_unit<CW, S>(pl.jobs, pl.tm, pl.tn, u, a.Gc, a.Phic, a.E_loc, a.K_cap, a.h, a.d, a.dW,
                     a.slots, ring_addr, acc);
#ifdef LRM_TIMELINE
    if (threadIdx.x == 0) stamp[1] = __builtin_amdgcn_s_memrealtime();
#endif
  }
  int u_dw = pl.j;
  bool dw_left = MIX, dx_left = true, dx_next = MIX;
  for (;;) {
    if (dw_left && !(dx_next && dx_left)) {
      const int32_t* jobs = pl.jobs;
      int u = u_dw;
      if constexpr (MIX) {
        if (threadIdx.x == 0) {
          const int G = a.sched[0];
          int v = atomicAdd(&a.queue[kMaxXcd], 1), g = 0;
          if (a.sched[3] == 2) {
            // claim v: tile v % tpe of the expert of rank v / tpe (largest first), found where
            // the snake deal put it: group g, job j of that group's list
            const int r = v / pl.tpe, n2 = 2 * G, q = r % n2;
            const int j = 2 * (r / n2) + (q >= G ? 1 : 0);
            g = r < a.E_loc ? (q < G ? q : n2 - 1 - q) : -1;
            v = j * pl.tpe + (v - r * pl.tpe);
          } else {
            // claim v: unit v - (units of the groups before g) of group g
            for (; g < G && g < kMaxXcd * kMaxGroupsPerXcd; ++g) {
              const int n = a.sched[4 + 3 * kMaxDwSlots + g] * pl.tpe;
              if (v < n) break;
              v -= n;
            }
            if (g >= G || g >= kMaxXcd * kMaxGroupsPerXcd) g = -1;
          }
          claimed[0] = g;
          claimed[1] = v;
        }
        __syncthreads();
        const int g = __builtin_amdgcn_readfirstlane(claimed[0]);
        u = __builtin_amdgcn_readfirstlane(claimed[1]);
        __syncthreads();
        if (g < 0) {
          dw_left = false;
#ifdef LRM_TIMELINE
          if (threadIdx.x == 0) stamp[1] = __builtin_amdgcn_s_memrealtime();
#endif
          continue;
        }
        jobs = a.sched + kDwHeader + (int64_t)g * dw_jobs_per_group(a.E_loc) * 4;
      } else {
        u_dw += pl.gs;
        dw_left = u_dw < pl.units;
      }
      dw_unit<CW, S>(jobs, pl.tm, pl.tn, u, a.Gc, a.Phic, a.E_loc, a.K_cap, a.h, a.d, a.dW,
                     a.slots, ring_addr, acc);
      dx_next = MIX;
#ifdef LRM_TIMELINE
      if (threadIdx.x == 0 && !dw_left) stamp[1] = __builtin_amdgcn_s_memrealtime();
#endif
      continue;
    }
    if (!dx_left) break;  // and no dW unit is left either
    if (threadIdx.x == 0) {
      int u = -1;
      for (int k = 0; k < a.nxcd && u < 0; ++k) {
        const int y = x + k < a.nxcd ? x + k : x + k - a.nxcd;
        const int lo = y * per, cnt = (lo + per < total ? lo + per : total) - lo;
        if (cnt <= 0) continue;
        const int v = atomicAdd(&a.queue[y], 1);
        if (v < cnt) u = lo + v;
      }
      *claimed = u;
    }
    __syncthreads();
    const int u = __builtin_amdgcn_readfirstlane(*claimed);
    __syncthreads();
    if (u < 0) {
      dx_left = false;
      continue;
    }
#ifdef LRM_TIMELINE
    if (threadIdx.x == 0 && claims < kTimelineUnits) {
      stamp[4 + 2 * claims] = __builtin_amdgcn_s_memrealtime();
      stamp[5 + 2 * claims] = (unsigned long long)u;
    }
    ++claims;
#endif
    dx_unit<CX, S>(a.Gc, a.W, a.cmp_off, a.tiles, u, a.K_cap, a.h, a.d, a.dphi, ring_addr, acc);
    dx_next = false;
  }
#ifdef LRM_TIMELINE
  if (threadIdx.x == 0) stamp[3] = (unsigned long long)claims;
#endif
}

// dW and dphi in one persistent launch (same tile shape, CW and CX differ only in the row
// operand's orientation), kPart 0.  Each workgroup runs its share of the dW units exactly as
// dw_bf16 does, then claims dphi units one at a time: from its own die's contiguous range (a
// counter per die in the workspace, reset by dx_schedule), and once that is exhausted from the
// other dies' in turn.  The workgroups whose dW share ends early (light groups) thus take more
// dphi units, and dphi's last partial round is spread over whoever is free.  A second launch of
// the same shape (kPart 1) follows it: for the products dw_schedule flags (fused_loop's MIX:
// store-bound, or an estimate that the dphi units should start first) the first launch returns
// at once and the second runs the product; otherwise the second adds the split experts' partial
// slots (dw_fixup's work) and returns.  Two specialised kernels instead of one with both loops
// keep the register allocation of the common path as it is.  With solo set (no second launch)
// the first launch runs every product the common way.  Each unit is computed whole by the
// workgroup that claims it, in the same order as in dx_bf16, so results do not depend on which
// workgroup runs it.  A claim tries every die once, so every workgroup leaves when all ranges are
// exhausted.
// kLayer (2: FC2, 1: FC1) only separates the two layers' launches in profiles.
template <class CW, class CX, int S, int kLayer, int kPart>
__global__ __launch_bounds__(CW::THREADS) void gemm_fused(
    const uint16_t* __restrict__ Gc, const uint16_t* __restrict__ Phic,
    const uint16_t* __restrict__ W, const int32_t* __restrict__ cmp_off,
    const int32_t* __restrict__ sched, const int32_t* __restrict__ tiles, int32_t* __restrict__ queue,
    int nxcd, int E_loc, int K_cap, int h, int d, float* __restrict__ dW,
    float* __restrict__ slots, float* __restrict__ dphi, int solo) {
  const FusedArgs a{Gc, Phic, W, cmp_off, sched, tiles, queue, nxcd, E_loc, K_cap, h, d, dW, slots,
                    dphi};
  static_assert(CW::BM == CX::BM && CW::BN == CX::BN && CW::THREADS == CX::THREADS, "one shape");
  static_assert(CW::MT == CX::MT && CW::NT == CX::NT, "one accumulator array for both");
  using R = Ring<CW, S>;
  static_assert(Ring<CX, S>::BYTES == R::BYTES, "one ring");
  const bool mix = a.sched[3] != 0 && !solo;
  if constexpr (kPart == 0) {
    if (mix) return;  // the second launch runs this product
  } else {
    if (!mix) {
      if (a.slots != nullptr)
        fixup_split_experts(a.sched, a.E_loc, a.h, a.d, a.slots, a.dW,
                            (int64_t)blockIdx.x * CW::THREADS + threadIdx.x,
                            (int64_t)gridDim.x * CW::THREADS);
      return;
    }
  }
  __shared__ __attribute__((aligned(1024))) uint16_t ring[R::BYTES / 2];
  // claimed units are broadcast through the ring's first two words: every mainloop ends with its
  // loads drained and a barrier, and the next one starts writing the ring only after the second
  // barrier of a claim
  volatile int* claimed = (volatile int*)ring;
  const uint32_t ring_addr = lds_addr(ring);
  unsigned long long* stamp = nullptr;
#ifdef LRM_TIMELINE
  stamp = g_timeline + (size_t)(blockIdx.x % kTimelineWGs) * kTimelineWords;
  if (threadIdx.x == 0) {
    stamp[0] = __builtin_amdgcn_s_memrealtime();
    stamp[1] = stamp[0];  // replaced when the last dW unit of this workgroup ends
    stamp[kTimelineWords - 4] = __builtin_amdgcn_s_memtime();
    stamp[kTimelineWords - 2] = __builtin_amdgcn_s_getreg((15 << 11) | 20);  // XCC_ID[15:0]
    stamp[kTimelineWords - 1] = __builtin_amdgcn_s_getreg((31 << 11) | 4);   // HW_ID[31:0]
  }
#endif
  f32x16 acc[CX::MT][CX::NT];
  fused_loop<CW, CX, S, kPart == 1>(a, claimed, ring_addr, acc, stamp);
#ifdef LRM_TIMELINE
  if (threadIdx.x == 0) {
    stamp[2] = __builtin_amdgcn_s_memrealtime();
    stamp[kTimelineWords - 3] = __builtin_amdgcn_s_memtime();
  }
#endif
}

// dW schedule (one workgroup, one thread per expert rank).  A job (one expert, or a piece of one
// along K) costs its K steps plus kDwJobCost (the fixed price of a job: the store of its fp32 tile,
// prologue and drain); G = nxcd * gpx groups share the total cost, T = ceil(total / G) each.
// Experts are ranked by retained rows (descending, ties by id).  Two plans:
//  * whole experts dealt to the groups in snake order (0..G-1, G-1..0, ..);
//  * when that leaves a group above 5T/4 and the slots suffice, a contiguous fill: the ranked
//    experts' costs are laid end to end and cut into G runs of T, an expert crossing a cut is
//    split there (cuts on K-step multiples, in proportion to its cost).  The first non-empty
//    piece writes dW, every later non-empty piece a partial slot that dw_fixup adds in piece
//    order; an empty piece is a skip record (slot -2).  An expert without rows writes zeros.
// Every step is a closed form or a workgroup scan, so the schedule costs a few barriers.
constexpr int kDwJobCost = 8;

// What the dW schedule needs to know of the one-launch form's dphi units (wgs = 0: no such form).
struct DxShape {
  int wgs;    // workgroups of the persistent grid
  int bm;     // rows per dphi unit
  int tn;     // column tiles per row tile
  int steps;  // K steps of a dphi unit
  int tpe;    // dW tiles per job
};

// The two orders of the one-launch form, estimated in K steps (a unit costs its steps plus
// kDwJobCost; a dW job's cost c covers each of its tpe tiles).  When its U dphi units fit in one
// round of the grid (U <= wgs, so each workgroup runs at most one):
//  * dW first: a workgroup's part of its group's load (share: the fill's T or the snake deal's
//    heaviest group), then one dphi unit;
//  * dphi first: the whole work spread over the grid, but no less than one dphi unit or the
//    costliest job, nor -- when more dW tiles than the free workgroups cost more than a dphi unit
//    -- than a dphi unit followed by the costliest job.
// With several rounds of dphi units both orders spread the same work; what differs is the end.
// Dynamic dphi claims after the dW shares end with the last dphi units, about half a unit after
// the mean (kd / 2); dphi first ends with dW tiles claimed largest expert first, which cost at
// most cmax.  dphi first is taken when the difference, (kd - cmax) / 2, exceeds 2 % of the
// spread work (it pays for the dW claims' looser L2 reuse).
// Thread r holds the rank-r expert's `rows` and cost `c`, cmax is the largest cost; every thread
// of the workgroup calls.  One scan sums both counts: row tiles in bits 0-19 (each expert's
// count capped at 1023, which still exceeds any grid, so the sum stays below 2^20), jobs longer
// than a dphi unit from bit 20 (at most E_loc <= 1024).
__device__ __forceinline__ bool dx_first_ends_sooner(const DxShape& dx, int rows, int c, int cmax,
                                                     int total, int share, int groups, int* sh) {
  const int kd = dx.steps + kDwJobCost;
  const int rt = (rows + dx.bm - 1) / dx.bm;
  int both = 0;
  block_exclusive_scan_1024((rt < 1023 ? rt : 1023) + (c > kd ? 1 << 20 : 0), sh, &both);
  const int row_tiles = both & ((1 << 20) - 1), nlong = both >> 20;
  const int64_t U = (int64_t)row_tiles * dx.tn, wgs = dx.wgs;
  if (U == 0) return false;
  if (U > wgs) {
    const int64_t spread = ((int64_t)total * dx.tpe + U * kd) / wgs;
    return (int64_t)(kd - cmax) * 25 > spread;
  }
  const int64_t gsz = wgs / groups;
  const int64_t dw_first = ((int64_t)share * dx.tpe + gsz - 1) / gsz + kd;
  int64_t dx_first = ((int64_t)total * dx.tpe + U * kd + wgs - 1) / wgs;
  dx_first = dx_first > kd ? dx_first : kd;
  dx_first = dx_first > cmax ? dx_first : cmax;
  if ((int64_t)nlong * dx.tpe > wgs - U && dx_first < kd + cmax) dx_first = kd + cmax;
  return dx_first < dw_first;
}

__device__ __forceinline__ void dw_schedule_body(const int32_t* __restrict__ cmp_off, int E_loc,
                                                 int K_cap, int groups, int gpx,
                                                 int32_t* __restrict__ sched, int allow_split,
                                                 const DxShape& dx) {
  constexpr int kG = kMaxXcd * kMaxGroupsPerXcd;
  __shared__ int rows[1024], by_rank[1024];
  __shared__ int load[kG], first[kG], count[kG];
  __shared__ int sh[40];
  __shared__ int cmax;
  const int tid = threadIdx.x;
  int mine = 0;
  if (tid < E_loc) {
    int a = cmp_off[tid], b = cmp_off[tid + 1];
    a = a < 0 ? 0 : (a > K_cap ? K_cap : a);
    b = b < a ? a : (b > K_cap ? K_cap : b);
    mine = b - a;
    rows[tid] = mine;
  }
  if (tid < kG) {
    load[tid] = 0;
    first[tid] = 0;
    count[tid] = 0;
  }
  __syncthreads();
  if (tid < E_loc) {
    int rank = 0;
    for (int y = 0; y < E_loc; ++y) {
      const int o = rows[y];
      rank += (o > mine) || (o == mine && y < tid);
    }
    by_rank[rank] = tid;
  }
  __syncthreads();
  // From here thread r handles the expert of rank r.
  const int r = tid;
  const int e = r < E_loc ? by_rank[r] : -1;
  int s = 0, n = 0;
  if (e >= 0) {
    s = cmp_off[e];
    s = s < 0 ? 0 : (s > K_cap ? K_cap : s);
    n = rows[e];
  }
  const int st = (n + kBK - 1) / kBK;
  const int c = e >= 0 ? st + kDwJobCost : 0;
  int total = 0;
  const int P = block_exclusive_scan_1024(c, sh, &total);
  const int T = total > 0 ? (total + groups - 1) / groups : 1;
  const int n2 = 2 * groups, q = r % n2, gs = q < groups ? q : n2 - 1 - q;
  if (e >= 0) atomicAdd(&load[gs], c);
  if (r == 0) cmax = c;  // rank 0 holds the most rows, so the costliest job
  __syncthreads();
  int worst = 0;
  for (int g = 0; g < groups; ++g) worst = load[g] > worst ? load[g] : worst;
  bool split_pays = allow_split && (int64_t)worst * 4 > (int64_t)T * 5 &&
                    groups - 1 <= kMaxDwSlots;
  if (split_pays && dx.wgs > 0) {
    // In the one-launch form the dphi units claimed after the dW shares absorb an uneven deal
    // when the heaviest group's share, per workgroup, stays within 3/4 of the work a workgroup
    // averages (dW and dphi spread over the grid): splitting would then only add the fix-up.
    int row_tiles = 0;
    const int rt = (e >= 0 ? n + dx.bm - 1 : 0) / dx.bm;
    block_exclusive_scan_1024(rt < 1023 ? rt : 1023, sh, &row_tiles);
    const int64_t spread = ((int64_t)total * dx.tpe +
                            (int64_t)row_tiles * dx.tn * (dx.steps + kDwJobCost)) / dx.wgs;
    const int64_t heavy = (int64_t)worst * dx.tpe / (dx.wgs / groups);
    if (heavy * 4 <= spread * 3) split_pays = false;
  }
  // dphi first (the second fused launch, with dynamic dW claims, which need no splits) when the
  // products are store-bound: the jobs' K steps (total - kDwJobCost * E_loc) sum to less than
  // their fixed costs; or when the one-launch form's dphi units fit in one round of the grid and
  // starting them first is estimated to end sooner
  // (flag 1: dW units claimed group by group, which spreads the heavy jobs among the light ones;
  // flag 2: largest expert first, so that the jobs longer than a dphi unit start at once)
  int mix = total - kDwJobCost * E_loc < kDwJobCost * E_loc ? 1 : 0;
  // a job of cost c holds more than 32 (c - kDwJobCost - 1) rows, so the dphi units number at
  // least tn * 32 * (total - (kDwJobCost + 1) * E_loc) / bm: when that exceeds the grid and no
  // job costs less than a dphi unit, the estimate cannot pick dphi first and is skipped
  if (!mix && dx.wgs > 0 &&
      ((int64_t)dx.tn * kBK * (total - (kDwJobCost + 1) * E_loc) <= (int64_t)dx.wgs * dx.bm ||
       cmax < dx.steps + kDwJobCost) &&
      dx_first_ends_sooner(dx, e >= 0 ? n : 0, c, cmax, total, split_pays ? T : worst, groups, sh))
    mix = 2;
  const bool fill = split_pays && !mix;
  const int64_t jpg = dw_jobs_per_group(E_loc);
  auto put = [&](int g, int idx, int kb, int kend, int slot) {
    int32_t* jb = sched + kDwHeader + (int64_t)g * jpg * 4 + 4 * idx;
    jb[0] = e;
    jb[1] = kb;
    jb[2] = kend;
    jb[3] = slot;
  };
  if (!fill) {
    // rank r is the (2 * (r / 2G) + [q >= G])-th job of its group
    if (e >= 0) put(gs, 2 * (r / n2) + (q >= groups ? 1 : 0), s, s + n, -1);
    if (tid < groups) {
      const int full = E_loc / n2, rem = E_loc % n2;
      count[tid] = 2 * full + (tid < rem ? 1 : 0) + (n2 - 1 - tid < rem ? 1 : 0);
    }
    if (tid == 0) sched[2] = 0;
  } else {
    // the run [P, P + c) meets groups g0..g1; a group's jobs are the ranks whose runs meet it
    const int g0 = P / T;
    int g1 = c > 0 ? (P + c - 1) / T : g0;
    g1 = g1 < groups - 1 ? g1 : groups - 1;
    if (e >= 0)
      for (int g = g0; g <= g1; ++g)
        if ((int64_t)g * T >= P) first[g] = r;  // this run holds the group's first cost unit
    // cut k (between piece k-1 and k) in K steps, proportional to the cost consumed before it
    auto cut = [&](int k) -> int {
      if (k == 0) return 0;
      if (k > g1 - g0) return st;
      const int64_t v = ((int64_t)(g0 + k) * T - P) * st / c;
      return (int)(v < 0 ? 0 : (v > st ? st : v));
    };
    int nonempty = 0, writer = -1;
    if (e >= 0)
      for (int k = 0; k <= g1 - g0; ++k)
        if (cut(k + 1) > cut(k)) {
          if (writer < 0) writer = k;
          ++nonempty;
        }
    if (writer < 0) writer = 0;
    const int need = nonempty > 1 ? nonempty - 1 : 0;
    int nslots = 0, nsplit = 0;
    const int slot0 = block_exclusive_scan_1024(need, sh, &nslots);
    const int rec = block_exclusive_scan_1024(need > 0 ? 1 : 0, sh, &nsplit);
    // the scans' barriers published first[]
    if (e >= 0) {
      int slot = slot0;
      for (int k = 0; k <= g1 - g0; ++k) {
        const int a = cut(k), b = cut(k + 1), g = g0 + k;
        const int kb = s + (a * kBK < n ? a * kBK : n), kend = s + (b * kBK < n ? b * kBK : n);
        put(g, r - first[g], kb, kend, k == writer ? -1 : (b > a ? slot++ : -2));
        atomicAdd(&count[g], 1);
      }
      if (need > 0) {
        sched[4 + 3 * rec] = e;
        sched[5 + 3 * rec] = slot0;
        sched[6 + 3 * rec] = need;
      }
    }
    if (tid == 0) sched[2] = nsplit;
  }
  __syncthreads();
  if (tid == 0) {
    sched[0] = groups;
    sched[1] = gpx;
    sched[3] = mix;
  }
  if (tid < groups) sched[4 + 3 * kMaxDwSlots + tid] = count[tid];
}

// ------------------------------------------------------------------------------------------------
// fp32 path (v_mfma_f32_32x32x2f32); LDS tiles are [k][mn] with a padded pitch.
// ------------------------------------------------------------------------------------------------
constexpr int FBM = 64, FBN = 64;    // workgroup tile: 4 wavefronts of 32 x 32
constexpr int BKF = 64;              // K per step
constexpr int PF = FBM + 4;          // floats per LDS k-row
constexpr int JF = BKF * FBM / 4 / 128;  // 16-byte chunks each of 128 threads moves per step
static_assert(FBM == FBN && FBM <= kDxTileM * 1 && kDxTileM == FBM, "dphi row tile of the table");

// [k][mn] source: BKF rows x 64 columns = 16 BKF chunks of 4 floats; thread t of 128 moves JF.
__device__ __forceinline__ void ld_kmn_f32(const float* __restrict__ X, int64_t ld, int k0,
                                           int kend, int mn0, int mnend, int t, float4 v[JF]) {
#pragma unroll
  for (int j = 0; j < JF; ++j) {
    const int c = t + 128 * j, row = c >> 4, col = mn0 + (c & 15) * 4;
    if (k0 + row < kend && col < mnend)
      v[j] = *(const float4*)(X + (int64_t)(k0 + row) * ld + col);
    else
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

__device__ __forceinline__ void st_kmn_f32(float* __restrict__ s, int t, const float4 v[JF]) {
#pragma unroll
  for (int j = 0; j < JF; ++j) {
    const int c = t + 128 * j, row = c >> 4, col = (c & 15) * 4;
    *(float4*)(s + row * PF + col) = v[j];
  }
}

// [mn][k] source: 64 rows x BKF k = 16 BKF chunks of 4 k; stored transposed into [k][mn].
__device__ __forceinline__ void ld_mnk_f32(const float* __restrict__ X, int64_t ld, int mn0,
                                           int mnend, int k0, int kend, int t, float4 v[JF]) {
#pragma unroll
  for (int j = 0; j < JF; ++j) {
    const int c = t + 128 * j, row = c / (BKF / 4), kc = (c % (BKF / 4)) * 4;
    if (mn0 + row < mnend && k0 + kc < kend)
      v[j] = *(const float4*)(X + (int64_t)(mn0 + row) * ld + k0 + kc);
    else
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

__device__ __forceinline__ void st_mnk_f32(float* __restrict__ s, int t, const float4 v[JF]) {
#pragma unroll
  for (int j = 0; j < JF; ++j) {
    const int c = t + 128 * j, row = c / (BKF / 4), kc = (c % (BKF / 4)) * 4;
    s[(kc + 0) * PF + row] = v[j].x;
    s[(kc + 1) * PF + row] = v[j].y;
    s[(kc + 2) * PF + row] = v[j].z;
    s[(kc + 3) * PF + row] = v[j].w;
  }
}

__device__ __forceinline__ void mma_step_f32(const float* __restrict__ sa,
                                             const float* __restrict__ sb, int wm, int wn,
                                             int lane, f32x16 acc[1][1]) {
  const int r = lane & 31, kh = lane >> 5;
#pragma unroll
  for (int ks = 0; ks < BKF; ks += 2) {
    const float a = sa[(ks + kh) * PF + wm * 32 + r];
    const float b = sb[(ks + kh) * PF + wn * 32 + r];
    acc[0][0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, acc[0][0], 0, 0, 0);
  }
}

// dW, fp32: one workgroup per 64 x 64 tile of one job.  Without a schedule (sched == nullptr) the
// job of blockIdx.z is expert blockIdx.z over its whole K range, written to dW.  With one,
// blockIdx.z walks dw_schedule's job lists group after group: an expert, or a piece of one along
// K whose partial sum goes to a slot that dw_fixup adds in piece order, so that one large expert
// no longer sets the end of the launch.
__global__ __launch_bounds__(kF32Threads) void dw_f32(const float* __restrict__ Gc,
                                                  const float* __restrict__ Phic,
                                                  const int32_t* __restrict__ cmp_off, int K_cap,
                                                  int h, int d, float* __restrict__ dW,
                                                  const int32_t* __restrict__ sched, int E_loc,
                                                  float* __restrict__ slots) {
  __shared__ __attribute__((aligned(16))) float sa[2][BKF * PF];
  __shared__ __attribute__((aligned(16))) float sb[2][BKF * PF];
  const int m0 = blockIdx.y * FBM, n0 = blockIdx.x * FBN;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;
  int e, s, t;
  float* out;
  if (sched == nullptr) {
    e = blockIdx.z;
    s = cmp_off[e];
    t = cmp_off[e + 1];
    s = s < 0 ? 0 : (s > K_cap ? K_cap : s);
    t = t < s ? s : (t > K_cap ? K_cap : t);
    out = dW + (int64_t)e * h * d;
  } else {
    const int G = sched[0];
    int z = blockIdx.z, g = 0;
    for (; g < G && g < kMaxXcd * kMaxGroupsPerXcd; ++g) {
      const int c = sched[4 + 3 * kMaxDwSlots + g];
      if (z < c) break;
      z -= c;
    }
    if (g >= G || g >= kMaxXcd * kMaxGroupsPerXcd) return;  // past the last job
    const int32_t* jb = sched + kDwHeader + (int64_t)g * dw_jobs_per_group(E_loc) * 4 + 4 * z;
    e = jb[0];
    s = jb[1];
    t = jb[2];
    const int slot = jb[3];
    if (slot == -2) return;  // an empty piece of a split expert
    // a record outside the buffers (never written so by dw_schedule) is skipped, not followed
    if (e < 0 || e >= E_loc || s < 0 || t < s || t > K_cap || slot < -1 || slot >= kMaxDwSlots)
      return;
    out = slot < 0 ? dW + (int64_t)e * h * d : slots + (int64_t)slot * h * d;
  }
  f32x16 acc[1][1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.0f;
  const bool isA = tid < 128;
  const int blk = tid & 127;
  const float* X = isA ? Gc : Phic;
  const int64_t ld = isA ? h : d;
  const int mn0 = isA ? m0 : n0, mnend = isA ? h : d;
  const int nk = (t - s + BKF - 1) / BKF;
  float4 v[JF];
  if (nk > 0) {
    ld_kmn_f32(X, ld, s, t, mn0, mnend, blk, v);
    st_kmn_f32(isA ? sa[0] : sb[0], blk, v);
  }
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < nk) ld_kmn_f32(X, ld, s + (kt + 1) * BKF, t, mn0, mnend, blk, v);
    mma_step_f32(sa[cur], sb[cur], wm, wn, lane, acc);
    if (kt + 1 < nk) st_kmn_f32(isA ? sa[cur ^ 1] : sb[cur ^ 1], blk, v);
    __syncthreads();
  }
  store_acc<1, 1, 2>(out, d, m0, h, n0, d, wm, wn, lane, acc);
}

// dphi, fp32: one workgroup per 64 x 64 tile of the tile table.  With fix_sched set (both products
// in one call, launched right after dw_f32) the workgroups first add the split experts' partial
// slots into dW, dw_fixup's work, which saves that launch when nothing is split.
__global__ __launch_bounds__(kF32Threads) void dx_f32(const float* __restrict__ Gc,
                                                  const float* __restrict__ W,
                                                  const int32_t* __restrict__ cmp_off,
                                                  const int32_t* __restrict__ tiles, int K_cap,
                                                  int h, int d, float* __restrict__ dphi,
                                                  const int32_t* __restrict__ fix_sched, int E_loc,
                                                  const float* __restrict__ slots,
                                                  float* __restrict__ dW) {
  __shared__ __attribute__((aligned(16))) float sa[2][BKF * PF];
  __shared__ __attribute__((aligned(16))) float sb[2][BKF * PF];
  if (fix_sched != nullptr)
    fixup_split_experts(fix_sched, E_loc, h, d, slots, dW,
                        ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kF32Threads + threadIdx.x,
                        (int64_t)gridDim.x * gridDim.y * kF32Threads);
  const int tile = blockIdx.x;
  if (tile >= tiles[0]) return;
  const int e = tiles[1 + 2 * tile], m0 = tiles[2 + 2 * tile];
  int mend = cmp_off[e + 1];
  mend = mend > K_cap ? K_cap : mend;
  const int n0 = blockIdx.y * FBN;
  const int tid = threadIdx.x, lane = lane_id(), wv = tid / kWave, wm = wv >> 1, wn = wv & 1;
  f32x16 acc[1][1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.0f;
  const bool isA = tid < 128;
  const int blk = tid & 127;
  const float* We = W + (int64_t)e * h * d;
  const int nk = (h + BKF - 1) / BKF;
  float4 v[JF];
  if (isA) {
    ld_mnk_f32(Gc, h, m0, mend, 0, h, blk, v);
    st_mnk_f32(sa[0], blk, v);
  } else {
    ld_kmn_f32(We, d, 0, h, n0, d, blk, v);
    st_kmn_f32(sb[0], blk, v);
  }
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    const int k1 = (kt + 1) * BKF;
    if (kt + 1 < nk) {
      if (isA) ld_mnk_f32(Gc, h, m0, mend, k1, h, blk, v);
      else ld_kmn_f32(We, d, k1, h, n0, d, blk, v);
    }
    mma_step_f32(sa[cur], sb[cur], wm, wn, lane, acc);
    if (kt + 1 < nk) {
      if (isA) st_mnk_f32(sa[cur ^ 1], blk, v);
      else st_kmn_f32(sb[cur ^ 1], blk, v);
    }
    __syncthreads();
  }
  store_acc<1, 1, 2>(dphi, d, m0, mend, n0, d, wm, wn, lane, acc);
}

// ------------------------------------------------------------------------------------------------
// dphi tile table: tiles[0] = number of row tiles, then (expert, first row) per tile, experts in
// order, `tm` rows per tile (the last tile of a segment is partial; empty segments have none).
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void dx_schedule_body(const int32_t* __restrict__ cmp_off, int E_loc,
                                                 int K_cap, int tm, int64_t max_tiles,
                                                 int32_t* __restrict__ tiles,
                                                 int32_t* __restrict__ queue) {
  __shared__ int sh[32];
  const int tid = threadIdx.x, w = tid / kWave, lane = lane_id();
  if (queue && tid <= kMaxXcd) queue[tid] = 0;  // unit counters of the fused launch (dphi per die, dW)
  int base_tiles = 0;
  for (int e0 = 0; e0 < E_loc; e0 += 1024) {
    const int e = e0 + tid;
    int s = 0, t = 0, nt = 0;
    if (e < E_loc) {
      s = cmp_off[e];
      t = cmp_off[e + 1];
      s = s < 0 ? 0 : (s > K_cap ? K_cap : s);
      t = t < s ? s : (t > K_cap ? K_cap : t);
      nt = (t - s + tm - 1) / tm;
    }
    const int inc = wave_inclusive_scan(nt);
    if (lane == kWave - 1) sh[w] = inc;
    __syncthreads();
    int before = base_tiles, total = base_tiles;
    for (int x = 0; x < 16; ++x) {
      if (x < w) before += sh[x];
      total += sh[x];
    }
    before += inc - nt;
    for (int j = 0; j < nt; ++j) {
      const int64_t idx = before + j;
      if (idx < max_tiles) {
        tiles[1 + 2 * idx] = e;
        tiles[2 + 2 * idx] = s + j * tm;
      }
    }
    base_tiles = total;
    __syncthreads();
  }
  if (tid == 0) tiles[0] = (int)(base_tiles < max_tiles ? base_tiles : max_tiles);
}

// dx: the one-launch form's dphi units of the same product, so that the separate dW call splits
// experts exactly when the one-launch form does and both give the same bits.
__global__ __launch_bounds__(1024) void dw_schedule(const int32_t* __restrict__ cmp_off, int E_loc,
                                                    int K_cap, int groups, int gpx,
                                                    int32_t* __restrict__ sched, DxShape dx) {
  dw_schedule_body(cmp_off, E_loc, K_cap, groups, gpx, sched, 1, dx);
}

__global__ __launch_bounds__(1024) void dx_schedule(const int32_t* __restrict__ cmp_off, int E_loc,
                                                    int K_cap, int tm, int64_t max_tiles,
                                                    int32_t* __restrict__ tiles,
                                                    int32_t* __restrict__ queue) {
  dx_schedule_body(cmp_off, E_loc, K_cap, tm, max_tiles, tiles, queue);
}

// Both schedules of the one-launch GEMMs in one launch of two workgroups: workgroup 0 builds the
// dW job lists, workgroup 1 the dphi tile table (and resets the unit counters); they write
// disjoint workspace regions.  allow_split = 0 keeps every expert whole (no partial slots).
__global__ __launch_bounds__(1024) void gemm_schedules(const int32_t* __restrict__ cmp_off,
                                                       int E_loc, int K_cap, int groups, int gpx,
                                                       int32_t* __restrict__ sched, int tm,
                                                       int64_t max_tiles,
                                                       int32_t* __restrict__ tiles,
                                                       int32_t* __restrict__ queue,
                                                       int allow_split, DxShape dx) {
  if (blockIdx.x == 0)
    dw_schedule_body(cmp_off, E_loc, K_cap, groups, gpx, sched, allow_split, dx);
  else
    dx_schedule_body(cmp_off, E_loc, K_cap, tm, max_tiles, tiles, queue);
}


// Persistent grid: one workgroup per CU (the 131-147 KiB of LDS per workgroup allows one), and the
// number of dies the workgroup ids are dealt over.
struct Grid {
  int blocks, nxcd;
};

Grid persistent_grid() {
  static int cus[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (cus[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cus[dev] = n;
  }
  const int n = cus[dev];
  const int nxcd = (n % kMaxXcd == 0 && n >= 8 * kMaxXcd) ? kMaxXcd : 1;
  return Grid{n / nxcd * nxcd, nxcd};
}

// Tile shapes.  Wide: 8 wavefronts (2 per SIMD), each 128 x 96, workgroup tile 256 x 384 -- the
// most output per byte staged (the L2-to-CU path, about 20 bytes per clock per CU, is what bounds
// these kernels).  Narrow fallbacks for d that 384-wide tiles would leave mostly empty.
using TileW_dW = Tile<4, 3, 4, true>;
using TileW_dX = Tile<4, 3, 4, false>;
using Tile192_dW = Tile<4, 3, 2, true>;
using Tile256_dW = Tile<4, 4, 2, true>;
using Tile128_dW = Tile<4, 2, 2, true>;
using Tile192_dX = Tile<4, 3, 2, false>;
using Tile256_dX = Tile<4, 4, 2, false>;
using Tile128_dX = Tile<4, 2, 2, false>;

// 0: 384-wide, 1: 256, 2: 192, 3: 128.  384 whenever at most a sixth of its columns would be
// empty; else the widest that divides d.
int pick_width(int d) {
  const int t384 = (d + 383) / 384;
  if (d >= 384 && t384 * 384 - d <= t384 * 64) return 0;
  if (d % 256 == 0) return 1;
  if (d % 192 == 0) return 2;
  return 3;
}

template <class C>
int groups_per_die(const lrm_problem& p, const Grid& g) {
  // as many groups per die as keep every group at least one job's tiles wide
  const int tpe = ((p.h + C::BM - 1) / C::BM) * ((p.d + C::BN - 1) / C::BN);
  const int nb = g.blocks / g.nxcd;
  for (int c = kMaxGroupsPerXcd; c > 1; c /= 2)
    if (nb % c == 0 && tpe * c <= nb) return c;
  return 1;
}

// The dphi units of the one-launch form on the same grid (its dphi tile has the dW tile's shape).
template <class C>
DxShape dx_shape(const lrm_problem& p, const Grid& g) {
  return DxShape{g.blocks, C::BM, (p.d + C::BN - 1) / C::BN, (p.h + kBK - 1) / kBK,
                 ((p.h + C::BM - 1) / C::BM) * ((p.d + C::BN - 1) / C::BN)};
}

template <class C>
void launch_dw_t(const lrm_problem& p, const void* Gc, const void* Phic, const int32_t* cmp_off,
                 int32_t* sched, float* dW, float* slots, const Grid& g, hipStream_t s) {
  const int gpx = groups_per_die<C>(p, g);
  hipLaunchKernelGGL(dw_schedule, dim3(1), dim3(kThreadsPerSchedule), 0, s, cmp_off, p.E_loc,
                     p.K_cap, g.nxcd * gpx, gpx, sched, dx_shape<C>(p, g));
  hipLaunchKernelGGL((dw_bf16<C, stages_for<C>()>), dim3(g.blocks), dim3(C::THREADS), 0, s,
                     (const uint16_t*)Gc, (const uint16_t*)Phic, sched, g.nxcd, p.E_loc, p.K_cap,
                     p.h, p.d, dW, slots);
  hipLaunchKernelGGL(dw_fixup, dim3(kFixupBlocks), dim3(256), 0, s, sched, p.E_loc,
                     p.h, p.d, slots, dW);
}

// slots == nullptr: experts are never split along K (no partial slots, no fix-up launch).
template <class CW, class CX, int kLayer>
void launch_fused_t(const lrm_problem& p, const void* Gc, const void* Phic, const void* W,
                    const int32_t* cmp_off, int32_t* sched, int32_t* tiles, int32_t* queue,
                    int64_t max_tiles, float* dW, float* slots, float* dphi, const Grid& g,
                    hipStream_t s) {
  const int gpx = groups_per_die<CW>(p, g);
  static_assert(kThreadsPerSchedule == 1024, "one block shape for both schedules");
  hipLaunchKernelGGL(gemm_schedules, dim3(2), dim3(1024), 0, s, cmp_off, p.E_loc, p.K_cap,
                     g.nxcd * gpx, gpx, sched, CX::BM, max_tiles, tiles, queue,
                     slots != nullptr ? 1 : 0, dx_shape<CW>(p, g));
  // without partial slots (the allocation-free entry) one launch runs every product
  const int solo = slots == nullptr ? 1 : 0;
  hipLaunchKernelGGL((gemm_fused<CW, CX, stages_for<CW>(), kLayer, 0>), dim3(g.blocks),
                     dim3(CW::THREADS), 0, s, (const uint16_t*)Gc, (const uint16_t*)Phic,
                     (const uint16_t*)W, cmp_off, sched, tiles, queue, g.nxcd, p.E_loc, p.K_cap,
                     p.h, p.d, dW, slots, dphi, solo);
  if (!solo)
    hipLaunchKernelGGL((gemm_fused<CW, CX, stages_for<CW>(), kLayer, 1>), dim3(g.blocks),
                       dim3(CW::THREADS), 0, s, (const uint16_t*)Gc, (const uint16_t*)Phic,
                       (const uint16_t*)W, cmp_off, sched, tiles, queue, g.nxcd, p.E_loc,
                       p.K_cap, p.h, p.d, dW, slots, dphi, 0);
}

template <class C>
void launch_dx_t(const lrm_problem& p, const void* Gc, const void* W, const int32_t* cmp_off,
                 const int32_t* tiles, float* dphi, const Grid& g, hipStream_t s) {
  hipLaunchKernelGGL((dx_bf16<C, stages_for<C>()>), dim3(g.blocks), dim3(C::THREADS), 0, s,
                     (const uint16_t*)Gc, (const uint16_t*)W, cmp_off, tiles, g.nxcd, p.K_cap, p.h,
                     p.d, dphi);
}

}  // namespace

hipError_t launch_dw(const lrm_problem& p, const void* Gc, const void* Phic, const int32_t* cmp_off,
                     float* dW, char* ws, const WsLayout& wl, hipStream_t s) {
  if (p.dtype == LRM_BF16) {
    const Grid g = persistent_grid();
    int32_t* sched = (int32_t*)(ws + wl.order);
    float* slots = (float*)(ws + wl.dwslots);
    switch (pick_width(p.d)) {
      case 0: launch_dw_t<TileW_dW>(p, Gc, Phic, cmp_off, sched, dW, slots, g, s); break;
      case 1: launch_dw_t<Tile256_dW>(p, Gc, Phic, cmp_off, sched, dW, slots, g, s); break;
      case 2: launch_dw_t<Tile192_dW>(p, Gc, Phic, cmp_off, sched, dW, slots, g, s); break;
      default: launch_dw_t<Tile128_dW>(p, Gc, Phic, cmp_off, sched, dW, slots, g, s); break;
    }
  } else {
    // kMaxXcd groups share the cost; the contiguous fill splits an expert above 5/4 of a share
    // into at most kMaxXcd - 1 extra pieces, so the jobs number at most E_loc + kMaxXcd - 1
    int32_t* sched = (int32_t*)(ws + wl.order);
    float* slots = (float*)(ws + wl.dwslots);
    hipLaunchKernelGGL(dw_schedule, dim3(1), dim3(kThreadsPerSchedule), 0, s, cmp_off, p.E_loc,
                       p.K_cap, kMaxXcd, 1, sched, DxShape{0, 1, 1, 0, 0});
    const dim3 grid((p.d + FBN - 1) / FBN, (p.h + FBM - 1) / FBM, p.E_loc + kMaxXcd - 1);
    hipLaunchKernelGGL(dw_f32, grid, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)Phic,
                       cmp_off, p.K_cap, p.h, p.d, dW, (const int32_t*)sched, p.E_loc, slots);
    hipLaunchKernelGGL(dw_fixup, dim3(kFixupBlocks), dim3(256), 0, s, sched, p.E_loc, p.h, p.d,
                       slots, dW);
  }
  return hipGetLastError();
}

hipError_t launch_dx(const lrm_problem& p, const void* Gc, const void* W, const int32_t* cmp_off,
                     float* dphi, char* ws, const WsLayout& wl, hipStream_t s) {
  int32_t* tiles = (int32_t*)(ws + wl.tiles);
  if (p.dtype == LRM_BF16) {
    const Grid g = persistent_grid();
    constexpr int BM = TileW_dX::BM;
    static_assert(BM == Tile128_dX::BM && BM >= kDxTileM, "one row tile for every width");
    const int64_t max_tiles = ((int64_t)p.K_cap + BM - 1) / BM + p.E_loc;
    hipLaunchKernelGGL(dx_schedule, dim3(1), dim3(1024), 0, s, cmp_off, p.E_loc, p.K_cap, BM,
                       max_tiles, tiles, nullptr);
    switch (pick_width(p.d)) {
      case 0: launch_dx_t<TileW_dX>(p, Gc, W, cmp_off, tiles, dphi, g, s); break;
      case 1: launch_dx_t<Tile256_dX>(p, Gc, W, cmp_off, tiles, dphi, g, s); break;
      case 2: launch_dx_t<Tile192_dX>(p, Gc, W, cmp_off, tiles, dphi, g, s); break;
      default: launch_dx_t<Tile128_dX>(p, Gc, W, cmp_off, tiles, dphi, g, s); break;
    }
  } else {
    hipLaunchKernelGGL(dx_schedule, dim3(1), dim3(1024), 0, s, cmp_off, p.E_loc, p.K_cap, FBM,
                       wl.max_tiles, tiles, nullptr);
    const dim3 grid((unsigned)wl.max_tiles, (p.d + FBN - 1) / FBN);
    hipLaunchKernelGGL(dx_f32, grid, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)W,
                       cmp_off, tiles, p.K_cap, p.h, p.d, dphi, (const int32_t*)nullptr, 0,
                       (const float*)nullptr, (float*)nullptr);
  }
  return hipGetLastError();
}

// The one-launch bf16 GEMMs on explicit schedule buffers (slots == nullptr: no expert splits).
template <int kLayer>
void launch_fused_bf16(const lrm_problem& p, const void* Gc, const void* Phic, const void* W,
                       const int32_t* cmp_off, float* dW, float* dphi, int32_t* sched,
                       int32_t* tiles, int32_t* queue, float* slots, hipStream_t s) {
  const Grid g = persistent_grid();
  static_assert(TileW_dX::BM == Tile128_dX::BM && TileW_dX::BM >= kDxTileM, "row tile");
  const int64_t max_tiles = ((int64_t)p.K_cap + TileW_dX::BM - 1) / TileW_dX::BM + p.E_loc;
  switch (pick_width(p.d)) {
    case 0:
      launch_fused_t<TileW_dW, TileW_dX, kLayer>(p, Gc, Phic, W, cmp_off, sched, tiles, queue,
                                            max_tiles, dW, slots, dphi, g, s);
      break;
    case 1:
      launch_fused_t<Tile256_dW, Tile256_dX, kLayer>(p, Gc, Phic, W, cmp_off, sched, tiles, queue,
                                            max_tiles, dW, slots, dphi, g, s);
      break;
    case 2:
      launch_fused_t<Tile192_dW, Tile192_dX, kLayer>(p, Gc, Phic, W, cmp_off, sched, tiles, queue,
                                            max_tiles, dW, slots, dphi, g, s);
      break;
    default:
      launch_fused_t<Tile128_dW, Tile128_dX, kLayer>(p, Gc, Phic, W, cmp_off, sched, tiles, queue,
                                            max_tiles, dW, slots, dphi, g, s);
      break;
  }
}

template <int kLayer>
hipError_t launch_gemms_t(const lrm_problem& p, const void* Gc, const void* Phic, const void* W,
                          const int32_t* cmp_off, float* dW, float* dphi, char* ws,
                          const WsLayout& wl, hipStream_t s) {
  if (p.dtype != LRM_BF16) {
    // fp32: both schedules in one launch, the dW jobs (experts split along K as the separate
    // call splits them), then the dphi tiles, whose workgroups first add the partial slots
    int32_t* sched = (int32_t*)(ws + wl.order);
    int32_t* tiles = (int32_t*)(ws + wl.tiles);
    float* slots = (float*)(ws + wl.dwslots);
    hipLaunchKernelGGL(gemm_schedules, dim3(2), dim3(1024), 0, s, cmp_off, p.E_loc, p.K_cap,
                       kMaxXcd, 1, sched, FBM, wl.max_tiles, tiles, (int32_t*)nullptr, 1,
                       DxShape{0, 1, 1, 0, 0});
    const dim3 gw((p.d + FBN - 1) / FBN, (p.h + FBM - 1) / FBM, p.E_loc + kMaxXcd - 1);
    hipLaunchKernelGGL(dw_f32, gw, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)Phic,
                       cmp_off, p.K_cap, p.h, p.d, dW, (const int32_t*)sched, p.E_loc, slots);
    const dim3 gx((unsigned)wl.max_tiles, (p.d + FBN - 1) / FBN);
    hipLaunchKernelGGL(dx_f32, gx, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)W,
                       cmp_off, tiles, p.K_cap, p.h, p.d, dphi, (const int32_t*)sched, p.E_loc,
                       (const float*)slots, dW);
    return hipGetLastError();
  }
  launch_fused_bf16<kLayer>(p, Gc, Phic, W, cmp_off, dW, dphi, (int32_t*)(ws + wl.order),
                            (int32_t*)(ws + wl.tiles), (int32_t*)(ws + wl.err) + kQueueWord,
                            (float*)(ws + wl.dwslots), s);
  return hipGetLastError();
}

hipError_t launch_gemms(const lrm_problem& p, const void* Gc, const void* Phic, const void* W,
                        const int32_t* cmp_off, float* dW, float* dphi, char* ws,
                        const WsLayout& wl, hipStream_t s, int layer) {
  return layer == 1 ? launch_gemms_t<1>(p, Gc, Phic, W, cmp_off, dW, dphi, ws, wl, s)
                    : launch_gemms_t<2>(p, Gc, Phic, W, cmp_off, dW, dphi, ws, wl, s);
}

// ------------------------------------------------------------------------------------------------
// Allocation-free variant of the FC2 GEMMs (lrm_grouped_dw_dx_noalloc).
//
// The only scratch the one-launch GEMMs need besides the caller's buffers is the schedule: the dW
// job lists, the dphi tile table and the per-die unit counters.  Here it lives in `scratch`, a
// file-scope device array of kNoallocScratchBytes that each GPU holds for the life of the
// process.  In host code `scratch` names a host-side stand-in; its device address on the current
// GPU is looked up once per device with hipGetSymbolAddress and only that address is passed to
// kernels.  Experts are never split along K in this variant (splitting needs h x d float32
// partial slots per split piece), so there is no fix-up launch.  Every call rewrites the schedule
// and the schedule kernel resets the counters; calls that overlap on one GPU share the array and
// race.
// ------------------------------------------------------------------------------------------------
static __device__ __align__(256) char scratch[kNoallocScratchBytes];

#ifdef LRM_TIMELINE
// Profiling builds only: copies the timestamp table (kTimelineWGs x kTimelineWords) to the host
// after the device is idle.
extern "C" int lrm_timeline_read(unsigned long long* host, size_t words) {
  if (words > (size_t)kTimelineWGs * kTimelineWords) return 1;
  if (hipDeviceSynchronize() != hipSuccess) return 2;
  return hipMemcpyFromSymbol(host, HIP_SYMBOL(g_timeline), words * 8, 0,
                             hipMemcpyDeviceToHost) != hipSuccess ? 3 : 0;
}
#endif

namespace {

std::mutex g_scratch_mu;
char* g_scratch_addr[kMaxDevices] = {};

hipError_t scratch_address(char** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_addr[dev] == nullptr) {
    void* ptr = nullptr;
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (ptr == nullptr) return hipErrorInvalidSymbol;
    g_scratch_addr[dev] = (char*)ptr;
  }
  *out = g_scratch_addr[dev];
  return hipSuccess;
}

}  // namespace

NoallocLayout noalloc_layout(const lrm_problem& p) {
  NoallocLayout l{};
  const int tm = p.dtype == LRM_BF16 ? TileW_dX::BM : FBM;
  l.max_tiles = ((int64_t)p.K_cap + tm - 1) / tm + p.E_loc;
  size_t off = 0;
  l.queue = off;
  off += 256;
  l.sched = off;
  off = align_up(off + (size_t)(kDwHeader + (int64_t)kMaxXcd * kMaxGroupsPerXcd *
                                             dw_jobs_per_group(p.E_loc) * 4) * 4, 256);
  l.tiles = off;
  off = align_up(off + (size_t)(1 + 2 * l.max_tiles) * 4, 256);
  l.total = off;
  return l;
}

hipError_t launch_gemms_noalloc(const lrm_problem& p, const void* Gc, const void* Phic,
                                const void* W, const int32_t* cmp_off, float* dW, float* dphi,
                                hipStream_t s) {
  const NoallocLayout l = noalloc_layout(p);
  if (l.total > kNoallocScratchBytes) return hipErrorInvalidValue;  // checked by the caller too
  char* base = nullptr;
  const hipError_t e = scratch_address(&base);
  if (e != hipSuccess) return e;
  int32_t* sched = (int32_t*)(base + l.sched);
  int32_t* tiles = (int32_t*)(base + l.tiles);
  int32_t* queue = (int32_t*)(base + l.queue);
  if (p.dtype == LRM_BF16) {
    launch_fused_bf16<2>(p, Gc, Phic, W, cmp_off, dW, dphi, sched, tiles, queue, nullptr, s);
  } else {
    const dim3 gw((p.d + FBN - 1) / FBN, (p.h + FBM - 1) / FBM, p.E_loc);
    hipLaunchKernelGGL(dw_f32, gw, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)Phic,
                       cmp_off, p.K_cap, p.h, p.d, dW, (const int32_t*)nullptr, p.E_loc,
                       (float*)nullptr);
    hipLaunchKernelGGL(dx_schedule, dim3(1), dim3(1024), 0, s, cmp_off, p.E_loc, p.K_cap, FBM,
                       l.max_tiles, tiles, nullptr);
    const dim3 gx((unsigned)l.max_tiles, (p.d + FBN - 1) / FBN);
    hipLaunchKernelGGL(dx_f32, gx, dim3(kF32Threads), 0, s, (const float*)Gc, (const float*)W,
                       cmp_off, tiles, p.K_cap, p.h, p.d, dphi, (const int32_t*)nullptr, 0,
                       (const float*)nullptr, (float*)nullptr);
  }
  return hipGetLastError();
}

}  // namespace lrm
