// dB_e[n][k] = sum over the rows r of expert e of D[r][n] A[r][k]: the weight
// gradient of the experts' product, A e4m3 with one e8m0 scale per 128 k of a
// row, D bf16 or in the same e4m3 form.
//
// The sum runs over the rows, and a scale belongs to a row: no scale of the
// scaled MFMA covers 32 of its values.  So elements are multiplied by their
// scales on the way to LDS, which is exact in bf16 (four bits of significand and a
// power of two), and v_mfma_f32_16x16x32_bf16 sums in fp32.  Both operands lie in
// LDS as they do in memory, rows r of columns, and are read transposed
// (ds_read_b64_tr_b16).
//
// Measured: 8192^3 802 us (1.37 PFLOP/s; a library product of bf16 reaches 1.41), with
// e4m3 D 817; 32768 rows of 16 experts x 4096 x 2048 525 and 500; 5000 rows of 8 x 1000 x
// 1408 with e4m3 D and a base 42.  Bound by the matrix cores together with LDS, which
// takes 512 cycles of writes and 1024 of reads for a slab's 2048 of MFMAs: without the
// conversions the time stays, without the LDS writes it falls by 5 to 10%, without the
// loads by 11 to 19%.
#include <atomic>
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "experts_device.hpp"
#include "fp8_rows.hpp"
#include "gemm_device.hpp"

namespace pgk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
#define PGK_INLINE __attribute__((always_inline))

constexpr int kThreads = 256;
constexpr int BR = 64;  // rows per slab: two steps of 32
constexpr int kRanked = 256;  // up to so many experts are taken in the order of their rows
constexpr int kScaleSlabs = 8, kScaleRows = kScaleSlabs * BR;  // a stretch of rows whose scales are fetched together

template <class F, int... I>
__device__ __forceinline__ void static_for_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_of(f, std::make_integer_sequence<int, N>{});
}

// Written out so that the accumulators stay in AGPRs (left to itself the register
// allocator moved them to VGPRs and spilled those).  The compiler's hazard logic does
// not look into it: a block's accumulator is next read NMF MFMAs later, the fragments
// come straight from LDS reads, which the compiler waits for, the accumulators are
// zeroed with padding after them, and read only after mfma_results_ready.
__device__ __forceinline__ void mfma16(f32x4& acc, bf16x8 a, bf16x8 b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// Zeros that are in their registers from here on: left to itself the compiler copied
// one set of them to each block right before its first MFMA.
__device__ __forceinline__ void zero_acc(f32x4& acc) {
  acc = f32x4{0, 0, 0, 0};
  asm volatile("" : "+a"(acc));
}

// Between the writes that zero the accumulators and the first MFMA that reads them.
__device__ __forceinline__ void acc_written() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Physical 16-byte chunk of logical chunk c in row r.  A transposing read of 32
// lanes touches rows r .. r + 3 and r + 8 .. r + 11 at two adjacent chunks: bits 2-3
// from r & 3 and bit 1 from bit 3 of r put those 16 chunks in distinct slots of a
// 256-byte window.  Bit 0 lets eight lanes, which the conversion has write every
// second chunk, meet the eight slots of a 128-byte one (bit 0 from bit 4 of the chunk: 8192^3
// of two e4m3 operands 827 us, so 817).
__device__ __forceinline__ int swz(int r, int c) {
  return c ^ (4 * (r & 3)) ^ (2 * ((r >> 3) & 1)) ^ (((c >> 3) ^ r) & 1);
}

// How an operand lies in memory: bf16 whose rows start on 16 bytes, bf16 of any
// alignment, or e4m3.
constexpr int kWide = 0, kNarrow = 1, kCodes = 2;
template <int W, int FORM>
struct Slab {
  static constexpr bool FP8 = FORM == kCodes;
  static constexpr int COLS = FP8 ? 16 : 8;          // of a part
  static constexpr int STEP = kThreads * COLS / W;   // rows from one part to the next
  static constexpr int PARTS = BR / STEP;
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int GROUPS = W / 128;
  // floats: the scales of two stretches of rows, the one in use and the next
  static constexpr int SCALES = FP8 ? 2 * GROUPS * kScaleRows : 0;
  static constexpr int FETCH = GROUPS * kScaleRows / kThreads;  // scale bytes per thread and stretch
  u32x4 q[PARTS];
  float sc[FP8 ? PARTS : 1];           // scales of the parts in q
  unsigned char fetched[FP8 ? FETCH : 1];
  float* scales;                       // LDS [2][GROUPS][kScaleRows]
  unsigned sc_at;                      // of part 0 of a slab, in floats
  unsigned off;                        // of part 0, in bytes
  unsigned wr[2];                      // LDS: FP8 its two chunks, else of even and odd parts
  unsigned long long x;                // the slab and its range
  unsigned xr;
  __device__ __forceinline__ void init(unsigned ld, float* lds) {
    const int c = (int)threadIdx.x % (W / COLS) * COLS, r = (int)threadIdx.x / (W / COLS), k = c >> 3;
    off = (unsigned)r * ld * ESZ + c * ESZ;
    scales = lds;
    sc_at = (unsigned)((c >> 7) * kScaleRows + r);
    wr[0] = (unsigned)(r * W * 2 + swz(r, k) * 16);
    wr[1] = FP8 ? (unsigned)(r * W * 2 + swz(r, k + 1) * 16) : (unsigned)((r + STEP) * W * 2 + swz(r + STEP, k) * 16);
  }
  // The slab from row r on, columns c0 .. of `cols`; left: rows from there to the
  // last (none: nothing is read).
  __device__ __forceinline__ void aim(int64_t r, int left, const void* mat, int64_t ld, int c0, int cols) {
    const int rows = left < BR ? left : BR;
    x = reinterpret_cast<unsigned long long>(mat) + (unsigned long long)(r * ld + c0) * ESZ;
    // up to the last column of the last row; what is loaded by words ends with a word
    xr = rows > 0 ? ((unsigned)(rows - 1) * (unsigned)ld + (unsigned)(cols - c0)) * ESZ : 0u;
    if (FORM == kWide) xr = (xr + 3u) & ~3u;
  }
  // Scale bytes of the stretch of rows r .. (left of them, the others zero) and groups
  // g0 .. of `groups`, and what they stand for into half `half`.
  __device__ __forceinline__ void fetch(const uint8_t* scale, int64_t sld, int64_t r, int left, int g0, int groups) {
    if (!FP8) return;
#pragma unroll
    for (int i = 0; i < FETCH; ++i) {
      const int at = i * kThreads + (int)threadIdx.x, row = at % kScaleRows, g = at / kScaleRows;
      fetched[FP8 ? i : 0] = row < left && g0 + g < groups ? scale[(int64_t)(g0 + g) * sld + r + row] : 0;
    }
  }
  __device__ __forceinline__ void keep(int half) {
    if (!FP8) return;
#pragma unroll
    for (int i = 0; i < FETCH; ++i)
      scales[half * GROUPS * kScaleRows + i * kThreads + (int)threadIdx.x] = scale_value(fetched[FP8 ? i : 0]);
  }
  // Part i of the slab aimed at, slab number s of the tile.
  __device__ __forceinline__ void load(int i, unsigned ld, int s) {
    const auto rX = rsrc(reinterpret_cast<const void*>(x), xr);
    // in the vector offset: the range check leaves a scalar one out
    const unsigned at = off + (unsigned)(i * STEP) * ld * ESZ;
    if (FORM != kNarrow) {
      q[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, at, 0, 0));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned lo = __builtin_amdgcn_raw_buffer_load_b16(rX, at + 4 * e, 0, 0);
        q[i][e] = lo | (unsigned)__builtin_amdgcn_raw_buffer_load_b16(rX, at + 4 * e + 2, 0, 0) << 16;
      }
    }
    if (FP8)
      sc[FP8 ? i : 0] = scales[(s / kScaleSlabs & 1) * GROUPS * kScaleRows + s % kScaleSlabs * BR + sc_at + i * STEP];
  }
  // What becomes of part i, as operations of an instruction or two each, which the main
  // loop spreads over its MFMAs.  Codes: eight times two values by their scale, which is exact in bf16;
  // two writes of eight values; the next slab's load.  bf16: the write and the load.  ld:
  // of the matrix, in elements; s: the next slab's number.
  static constexpr int OPS = FP8 ? 11 : 2;  // per part
  u32x4 lo, hi;                             // the part under conversion
  template <int OP>
  __device__ __forceinline__ void run(unsigned char* st, unsigned ld, int s) {
    constexpr int i = OP / OPS, o = OP % OPS;
    if constexpr (!FP8) {
      if constexpr (o == 0)
        *reinterpret_cast<u32x4*>(st + wr[i & 1] + (i & ~1) * STEP * W * 2) = q[i];
      else
        load(i, ld, s);
    } else if constexpr (o < 8) {
      const unsigned w = q[i][o >> 1];
      const unsigned v =
          __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, sc[i], (o & 1) != 0));
      if constexpr (o < 4)
        lo[o] = v;
      else
        hi[o - 4] = v;
    } else if constexpr (o < 10) {
      *reinterpret_cast<u32x4*>(st + wr[o - 8] + i * STEP * W * 2) = o == 8 ? lo : hi;
    } else {
      load(i, ld, s);
    }
  }
};

// A tile is BN x BK of one expert's gradient; four waves of BN/2 x BK/2.
//
// Slabs go from memory to registers, are multiplied by their scales there and
// written to one of two LDS stages while the matrix cores work on the other; a part's
// next load goes out as soon as it is written, a whole period before it is needed.  One
// barrier per slab, between its two steps: behind it the second step's fragments are in
// registers already and the next slab's first are read.  Scales come by stretches of 512
// rows, a byte or two per thread, and lie in LDS as floats: a byte load beside every
// part's own cost as much as the conversions and the LDS writes (8192^3 863 us, without 811).
//
// A workgroup takes one tile: a tile's time goes with its expert's rows, which only
// the device knows, and the hardware hands the next workgroup to the next free CU.
template <int BN, int BK, int DFORM, bool F32>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(WgradParams p) {
  constexpr int TN = BN / 2, TK = BK / 2, SN = TN / 16, SK = TK / 16, NMF = SN * SK;
  constexpr int D_BYTES = BR * BN * 2, STAGE = D_BYTES + BR * BK * 2;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];  // [2][STAGE], D's scales, A's
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wk = wave & 1;
  const int npn = (p.N + BN - 1) / BN, npk = (p.K + BK - 1) / BK, per = npn * npk;
  const int np = (p.N + 127) / 128 * 128, kp = (p.K + 127) / 128 * 128;

  // The tile.  Workgroups go to the XCDs in turn, so that each XCD gets an equal part
  // of every expert, a compact block of its tiles whose operand panels meet in the
  // XCD's L2; and the experts with the most rows come first, so that the last
  // workgroups are short.
  __shared__ int s_rows[kRanked];
  int e = (int)(blockIdx.x / (unsigned)per);
  if (p.experts <= kRanked) {
    for (int i = tid; i < p.experts; i += kThreads) s_rows[i] = expert_rows(p.offsets, i, p.rows).n;
    __syncthreads();
    int* s_e = reinterpret_cast<int*>(smem);
    for (int i = tid; i < p.experts; i += kThreads) {
      const int n = s_rows[i];
      int before = 0;
      for (int j = 0; j < p.experts; ++j) before += s_rows[j] > n || (s_rows[j] == n && j < i) ? 1 : 0;
      if (before == e) *s_e = i;
    }
    __syncthreads();
    e = *s_e;
    __syncthreads();
  }
  e = __builtin_amdgcn_readfirstlane(e);
  int i_tile = (int)(blockIdx.x % (unsigned)per);
  if (p.xcds > 1 && per % p.xcds == 0) i_tile = i_tile % p.xcds * (per / p.xcds) + i_tile / p.xcds;
  int pn, pk;
  pgs::decode(pgs::kGrouped, i_tile, npn, npk, 8, pn, pk);
  const int n0 = __builtin_amdgcn_readfirstlane(pn) * BN, k0 = __builtin_amdgcn_readfirstlane(pk) * BK;
  const ExpertRows rows = expert_rows(p.offsets, e, p.rows);
  const int lo = __builtin_amdgcn_readfirstlane(rows.lo), n_rows = __builtin_amdgcn_readfirstlane(rows.n);

  Slab<BN, DFORM> d;
  Slab<BK, kCodes> a;
  constexpr int PD = Slab<BN, DFORM>::PARTS, PA = Slab<BK, kCodes>::PARTS, NP = PD + PA;
  const unsigned ldd = (unsigned)p.ldd;
  float* const s_scales = reinterpret_cast<float*>(smem + 2 * STAGE);
  d.init(ldd, s_scales);
  a.init((unsigned)kp, s_scales + Slab<BN, DFORM>::SCALES);
  // The loads are at slab number `at`.
  int at = 0;
  auto load = [&](int i) PGK_INLINE {
    if (i < PD)
      d.load(i, ldd, at);
    else
      a.load(i - PD, (unsigned)kp, at);
  };
  auto aim = [&]() {
    const int64_t r0 = (int64_t)at * BR;
    d.aim(lo + r0, (int)(n_rows - r0), p.D, p.ldd, n0, DFORM == kCodes ? np : p.N);
    a.aim(lo + r0, (int)(n_rows - r0), p.A, kp, k0, kp);
  };
  auto fetch = [&](int stretch) {
    const int64_t r0 = (int64_t)stretch * kScaleRows;
    d.fetch(p.sd, p.rows, lo + r0, (int)(n_rows - r0), n0 >> 7, np >> 7);
    a.fetch(p.sa, p.rows, lo + r0, (int)(n_rows - r0), k0 >> 7, kp >> 7);
  };
  auto keep = [&](int stretch) {
    d.keep(stretch & 1);
    a.keep(stretch & 1);
  };

  // Operation o of the slab that the registers hold, into the stage at s.
  constexpr int OD = PD * Slab<BN, DFORM>::OPS, OPS = OD + PA * Slab<BK, kCodes>::OPS;
  auto run = [&](auto oc, unsigned char* s) PGK_INLINE {
    constexpr int o = oc;
    if constexpr (o < OD)
      d.template run<o>(s, ldd, at);
    else
      a.template run<o - OD>(s + D_BYTES, (unsigned)kp, at);
  };

  // Fragments: lane i of a group of 16 points at row i / 4 (+ 8 per group), columns
  // 4 (i % 4) .. of a block, and receives four rows of column i.
  const int g4 = lane >> 4, i16 = lane & 15, a4 = i16 & 3, e4 = i16 >> 2;
  const int rl = g4 * 8 + e4;
  unsigned rd_d[SN], rd_a[SK];  // + 4 and 32 rows: the swizzle is unchanged
#pragma unroll
  for (int j = 0; j < SN; ++j) rd_d[j] = (unsigned)(rl * BN * 2 + swz(rl, (wn * TN + j * 16 + 4 * a4) >> 3) * 16 + 8 * (a4 & 1));
#pragma unroll
  for (int j = 0; j < SK; ++j)
    rd_a[j] = (unsigned)(D_BYTES + rl * BK * 2 + swz(rl, (wk * TK + j * 16 + 4 * a4) >> 3) * 16 + 8 * (a4 & 1));
  i16x4 fd[2][SN][2], fa[2][SK][2];
  constexpr int NR = 2 * (SN + SK);
  auto read = [&](const unsigned char* s, auto hc, int i) PGK_INLINE {
    constexpr int h = hc;  // step
    const int j = i >> 1, q = i & 1;
    // swz(r + 4, c) and swz(r, c) agree: r & 3, bit 3 and bit 0 do (r % 8 is below 4)
    if (j < SK)
      fa[h][j][q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(s + rd_a[j] + (h * 32 + q * 4) * BK * 2));
    else
      fd[h][j - SK][q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(s + rd_d[j - SK] + (h * 32 + q * 4) * BN * 2));
  };
  f32x4 acc[SN][SK];
  auto mfma = [&](auto hc, auto jc) PGK_INLINE {
    constexpr int h = hc, x = jc / SK, y = jc % SK;
    const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(fa[h][y][0], fa[h][y][1], 0, 1, 2, 3, 4, 5, 6, 7));
    const bf16x8 vd = __builtin_bit_cast(bf16x8, __builtin_shufflevector(fd[h][x][0], fd[h][x][1], 0, 1, 2, 3, 4, 5, 6, 7));
    mfma16(acc[x][y], va, vd);
  };

  // Lane: row n of the block i16, columns k 4 g4 .. + 3.  The base's blocks of a row of
  // blocks are loaded before the row before it is stored: base may be dB, so that the
  // compiler keeps loads behind stores as they are written (5000 rows of 8 x 1000 x 1408
  // with a base, one block after the other 52.1 us, so 43.1).
  typedef std::conditional_t<F32, float, unsigned short> out_t;
  auto store = [&]() {
    const int n = n0 + wn * TN + i16, k = k0 + wk * TK + 4 * g4;
    const int64_t at = ((int64_t)e * p.N + n) * p.K + k;
    out_t* out = static_cast<out_t*>(p.dB) + at;
    const out_t* base = static_cast<const out_t*>(p.base) + at;
    f32x4 held[2][SK];
    auto load_base = [&](int i) PGK_INLINE {
#pragma unroll
      for (int j = 0; j < SK; ++j) {
        const out_t* b = base + (int64_t)i * 16 * p.K + j * 16;
        const int cols = n + i * 16 < p.N ? p.K - k - j * 16 : 0;
        f32x4 v = {0, 0, 0, 0};
        if (cols >= 4) {
          if constexpr (F32) {
            v = __builtin_bit_cast(f32x4, (u32x4)*reinterpret_cast<const u32x4_a4*>(b));
          } else {
            const u32x2 w = *reinterpret_cast<const u32x2_a2*>(b);
            v = f32x4{__builtin_bit_cast(float, w[0] << 16), __builtin_bit_cast(float, w[0] & 0xffff0000u),
                      __builtin_bit_cast(float, w[1] << 16), __builtin_bit_cast(float, w[1] & 0xffff0000u)};
          }
        } else {
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            if (q >= cols) continue;
            if constexpr (F32)
              v[q] = b[q];
            else
              v[q] = __builtin_bit_cast(float, (unsigned)b[q] << 16);
          }
        }
        held[i & 1][j] = v;
      }
    };
    if (p.base) load_base(0);
#pragma unroll
    for (int i = 0; i < SN; ++i) {
      if (p.base && i + 1 < SN) load_base(i + 1);
#pragma unroll
      for (int j = 0; j < SK; ++j) {
        out_t* o = out + (int64_t)i * 16 * p.K + j * 16;
        const int cols = n + i * 16 < p.N ? p.K - k - j * 16 : 0;
        f32x4 v = {acc_read(acc[i][j][0]), acc_read(acc[i][j][1]), acc_read(acc[i][j][2]), acc_read(acc[i][j][3])};
        if (p.base) v += held[i & 1][j];
        if (cols >= 4) {
          if constexpr (F32)
            *reinterpret_cast<u32x4_a4*>(o) = __builtin_bit_cast(u32x4, v);
          else
            *reinterpret_cast<u32x2_a2*>(o) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            if (q >= cols) continue;
            if constexpr (F32)
              o[q] = v[q];
            else
              o[q] = (unsigned short)pack_bf16x2(v[q], v[q]);
          }
        }
      }
    }
  };

  const std::integral_constant<int, 0> step0;
  const std::integral_constant<int, 1> step1;
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SK; ++j) zero_acc(acc[i][j]);
  acc_written();
  // Step h of a slab on the matrix cores, among them the LDS reads of the next step (of
  // the stage at `from`) and this half of a period's operations (into the stage at `to`).
  // The second step comes first in a period.
  auto step = [&](auto hc, const unsigned char* from, unsigned char* to, auto both) PGK_INLINE {
    static_for<NMF>([&](auto jc) PGK_INLINE {
      constexpr int h = hc, j = jc, at = both ? (1 - h) * NMF + j : j, all = both ? 2 * NMF : NMF;
      mfma(hc, jc);
      constexpr int r0 = (j * NR + NMF - 1) / NMF, r1 = ((j + 1) * NR + NMF - 1) / NMF;
      static_for<r1 - r0>([&](auto rc) PGK_INLINE { read(from, std::integral_constant<int, 1 - h>{}, r0 + rc); });
      constexpr int o0 = (at * OPS + all - 1) / all, o1 = ((at + 1) * OPS + all - 1) / all;
      static_for<o1 - o0>([&](auto oc) PGK_INLINE { run(std::integral_constant<int, o0 + oc>{}, to); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  const std::integral_constant<bool, true> shared;
  const std::integral_constant<bool, false> alone;
  if (n_rows > 0) {
    unsigned char* const stage0 = smem;
    unsigned char* const stage1 = smem + STAGE;
    fetch(0);
    keep(0);
    fetch(1);
    keep(1);
    slab_barrier();
    aim();
#pragma unroll
    for (int i = 0; i < NP; ++i) load(i);
    ++at;
    aim();
    static_for<OPS>([&](auto oc) PGK_INLINE { run(oc, stage0); });
    ++at;
    aim();
    slab_barrier();
#pragma unroll
    for (int i = 0; i < NR; ++i) read(stage0, step0, i);
    __builtin_amdgcn_sched_barrier(0);
    step(step0, stage0, stage1, alone);
    slab_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // A period: the second step of slab s, then the first of slab s + 1, whose stage
    // is complete; slab s + 2 goes where slab s was, which no wave reads any more, and
    // slab s + 3, `at`, is loaded.  Where that is the second of a stretch, the scales of
    // the stretch after take the place of those of the one before, which the slab before
    // it was the last to read in another period.
    for (int s = 0; (int64_t)(s + 1) * BR < n_rows; ++s) {
      unsigned char* now = s & 1 ? stage1 : stage0;
      unsigned char* next = s & 1 ? stage0 : stage1;
      ++at;
      aim();
      const bool turn = at % kScaleSlabs == 1 && at > 1;
      if (turn) fetch(at / kScaleSlabs + 1);
      step(step1, next, now, shared);
      step(step0, next, now, shared);
      if (turn) keep(at / kScaleSlabs + 1);
      slab_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
    static_for<NMF>([&](auto jc) PGK_INLINE { mfma(step1, jc); });
  }
  mfma_results_ready();
  store();
}

// A built tile: its kernel and dynamic LDS; the limit of the latter is raised once per
// device.
constexpr int kDevices = 64;
struct Instance {
  int bn, bk, lds;
  void (*kern)(WgradParams);
  mutable std::atomic<bool> ready[kDevices] = {};
  hipError_t launch(const WgradParams& p, hipStream_t stream) const {
    int dev = 0;
    const bool known = hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kDevices;
    if (!known || !ready[dev].load(std::memory_order_acquire)) {
      (void)hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (known) ready[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (int64_t)p.experts * ((p.N + bn - 1) / bn) * ((p.K + bk - 1) / bk);
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(kThreads), lds, stream, p);
    return hipGetLastError();
  }
};
template <int BN, int BK, int DFORM, bool F32>
Instance tiled() {
  return {BN, BK, 2 * BR * (BN + BK) * 2 + 4 * (Slab<BN, DFORM>::SCALES + Slab<BK, kCodes>::SCALES),
          wgrad_kernel<BN, BK, DFORM, F32>};
}

}  // namespace

// Tiles of 256 x 256 where they give every CU one and do not cover half as much again as
// tiles of 128 x 128 (of 128 columns they leave half empty).  us, 256 x 256 / 128 x 128, whole
// tiles: 32768 rows of 16 experts x 4096 x 2048 523 / 678, 8192 of 4 x 2048 x 2048 69 / 91, of 64 x
// 256 x 2048 44 / 49.  A third more: 32768 of 16 x 300 x 2048 70 / 74, 8192 of 64 x 300 x 1024 42 /
// 37, of 32 x 1152 x 640 (e4m3) 45 / 39.  Twice as much: 8192 of 64 x 128 x 2048 40 / 26, 32768
// (e4m3) 60 / 42.  Fewer tiles than CUs: 8192 of 3 x 2048 x 2048 76 / 83, of 8 x 1000 x 1408 39 /
// 40, 5000 (e4m3) 31.3 / 30.7.
hipError_t launch_gemm_experts_wgrad(const WgradParams& p, int cus, hipStream_t stream) {
  static const Instance big[2][2] = {{tiled<256, 256, kWide, false>(), tiled<256, 256, kWide, true>()},
                                     {tiled<256, 256, kCodes, false>(), tiled<256, 256, kCodes, true>()}};
  static const Instance small[3][2] = {{tiled<128, 128, kWide, false>(), tiled<128, 128, kWide, true>()},
                                       {tiled<128, 128, kCodes, false>(), tiled<128, 128, kCodes, true>()},
                                       {tiled<128, 128, kNarrow, false>(), tiled<128, 128, kNarrow, true>()}};
  const int64_t tiles = (int64_t)p.experts * ((p.N + 255) / 256) * ((p.K + 255) / 256);
  const int64_t quarters = (int64_t)p.experts * ((p.N + 127) / 128) * ((p.K + 127) / 128);
  const int f32 = p.out_f32 ? 1 : 0;
  if (!p.sd && ((reinterpret_cast<uintptr_t>(p.D) & 15) != 0 || (p.ldd & 7) != 0)) return small[2][f32].launch(p, stream);
  return (tiles >= cus && 8 * tiles < 3 * quarters ? big : small)[p.sd ? 1 : 0][f32].launch(p, stream);
}

}  // namespace pgk
