// C[r][n] = sum over k of A[r][k] B_e[n][k], e the expert of row r: A e4m3 with
// one e8m0 scale per 128 k of a row, B e4m3 with one per block of 128 n x 128 k,
// fp32 accumulate, C bf16 or fp32.
//
// To bf16 the products run on the scaled e4m3 MFMA.  It keeps a product to 2^-13
// of the largest of eight that it adds first (measured: 2^2 beside 2^16 is lost
// there, 2^3 is not).  A result's error was 1.5e-5 of its size at random signs and any K,
// which bf16's own 2^-8 hides: the distance from 64 bits is that of an fp32 sum rounded to
// bf16 (1.7e-3 of the norm both), though one or two results in a hundred round the other
// way (3.4e-4 of the norm between the two).  Where terms cancel it is not hidden: the bound is
// 2^-10 of the sum of the terms' magnitudes.  To fp32 the elements are multiplied by
// their scales, exactly, into bf16 and go through the bf16 MFMA, which adds their exact
// products in fp32 at half the rate.
//
// The rows are sorted by expert and the experts' row counts are in device memory:
// each program of the grid adds up the tiles that the experts have and walks the
// tiles with a stride of the grid.
#include <atomic>
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "experts_device.hpp"
#include "fp8_rows.hpp"
#include "gemm_device.hpp"

namespace pgk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef unsigned u32_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

constexpr int kFmtE4M3 = 0;  // f8f6f4 operand format code of e4m3
#define PGK_INLINE __attribute__((always_inline))

// Columns n .. n + 3 of a row of C that ends at N.
__device__ __forceinline__ void store4(void* C, bool f32, int64_t at, int64_t n, int64_t N, f32x4 v) {
  if (f32) {
    float* p = static_cast<float*>(C) + at + n;
    if (n + 4 <= N) {
      *reinterpret_cast<u32x4_a4*>(p) = __builtin_bit_cast(u32x4, v);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (n + e < N) p[e] = v[e];
    }
  } else {
    unsigned short* p = static_cast<unsigned short*>(C) + at + n;
    const unsigned lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (n + 4 <= N) {
      *reinterpret_cast<u32x2_a2*>(p) = u32x2{lo, hi};
    } else {
      if (n < N) p[0] = (unsigned short)lo;
      if (n + 1 < N) p[1] = (unsigned short)(lo >> 16);
      if (n + 2 < N) p[2] = (unsigned short)hi;
    }
  }
}

// 32 codes of a lane (two pieces of 16) times their scale, as four operands of
// v_mfma_f32_16x16x32_bf16.
struct Exact {
  bf16x8 v[4];
  __device__ __forceinline__ Exact(const u32x4 (&q)[2], float scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned w = q[i >> 1][2 * (i & 1) + h];
        o[2 * h] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, false));
        o[2 * h + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, true));
      }
      v[i] = __builtin_bit_cast(bf16x8, o);
    }
  }
};

// ------------------------------------------------------------- few rows each
//
// A tile is 16 * SM rows by 16 * SN columns on v_mfma_scale_f32_16x16x128: one
// instruction takes one scale group of k.  The waves of a workgroup split K, keep
// DEPTH groups of their stretch in flight and add their sums in LDS.
template <int SM, int SN, int DEPTH, int WAVES, bool F32>
__global__ void __launch_bounds__(WAVES * 64) gemm_experts_stream_kernel(ExpertsParams p) {
  __shared__ f32x4 s_part[2][WAVES][SN][SM][64];
  extern __shared__ int s_experts[];
  int* s_lo = s_experts;
  int* s_n = s_lo + p.experts;
  int* s_tile = s_n + p.experts;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kb = lane >> 4;
  const int npn = (p.N + 16 * SN - 1) / (16 * SN);
  expert_tiles(p.offsets, p.experts, p.rows, 16 * SM, npn, s_lo, s_n, s_tile);
  const int total = s_tile[p.experts];
  const int groups = p.K >> 7, nb = (p.N + 127) >> 7;
  const int u0 = groups * wave / WAVES, u1 = groups * (wave + 1) / WAVES;
  struct Unit {
    u32x4 a[SM][2], b[SN][2];
    unsigned sa[SM], sb;
  };
  int e = 0, turn = 0;
  for (int t = blockIdx.x; t < total; t += gridDim.x, turn ^= 1) {
    e = __builtin_amdgcn_readfirstlane(expert_of_tile(s_tile, p.experts, t, e));
    const int lo = __builtin_amdgcn_readfirstlane(s_lo[e]), n_rows = __builtin_amdgcn_readfirstlane(s_n[e]);
    const int i = t - __builtin_amdgcn_readfirstlane(s_tile[e]);
    // the row tiles of one stretch of columns one after the other
    const int npm = (n_rows + 16 * SM - 1) / (16 * SM);
    const int m0 = i % npm * 16 * SM, n0 = i / npm * 16 * SN;
    const int ra = n_rows - m0 < 16 * SM ? n_rows - m0 : 16 * SM, rb = p.N - n0 < 16 * SN ? p.N - n0 : 16 * SN;
    const auto rA = rsrc(p.A + ((int64_t)lo + m0) * p.K, (unsigned)(ra * p.K));
    const auto rB = rsrc(p.B + ((int64_t)e * p.N + n0) * p.K, (unsigned)(rb * p.K));
    const uint8_t* sb = p.sb + ((int64_t)e * nb + (n0 >> 7)) * groups;
    const unsigned off = (unsigned)l16 * (unsigned)p.K + (unsigned)kb * 16u;
    auto load = [&](int u, Unit& x) PGK_INLINE {
      const auto rS = rsrc(p.sa + (int64_t)u * p.rows + lo + m0, (unsigned)ra);
#pragma unroll
      for (int j = 0; j < SN; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x.b[j][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rB, off + (unsigned)(j * 16) * (unsigned)p.K + (unsigned)(u * 128 + h * 64), 0, 0));
#pragma unroll
      for (int m = 0; m < SM; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x.a[m][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              rA, off + (unsigned)(m * 16) * (unsigned)p.K + (unsigned)(u * 128 + h * 64), 0, 0));
        x.sa[m] = __builtin_amdgcn_raw_buffer_load_b8(rS, (unsigned)(m * 16 + l16), 0, 0);
      }
      x.sb = sb[u];
    };
    f32x4 acc[SN][SM] = {};
    Unit x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (u0 + d < u1) load(u0 + d, x[d]);
    for (int u = u0; u < u1; u += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (u + d >= u1) break;
        if constexpr (F32) {
          const float sb_value = scale_value(x[d].sb);
#pragma unroll
          for (int m = 0; m < SM; ++m) {
            const Exact a(x[d].a[m], scale_value(x[d].sa[m]));
#pragma unroll
            for (int j = 0; j < SN; ++j) {
              const Exact b(x[d].b[j], sb_value);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[j][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], acc[j][m], 0, 0, 0);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < (F32 ? 0 : SN); ++j)
#pragma unroll
          for (int m = 0; m < SM; ++m) {
            const u32x4 b0 = x[d].b[j][0], b1 = x[d].b[j][1], a0 = x[d].a[m][0], a1 = x[d].a[m][1];
            acc[j][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                i32x8{(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]},
                i32x8{(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]},
                acc[j][m], kFmtE4M3, kFmtE4M3, 0, (int)x[d].sb, 0, (int)x[d].sa[m]);
          }
        if (u + DEPTH + d < u1) load(u + DEPTH + d, x[d]);
      }
    }
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int m = 0; m < SM; ++m) s_part[turn][wave][j][m][lane] = acc[j][m];
    // the sums of the tile before were read before this barrier, so that two
    // sets are enough
    __syncthreads();
    for (int q = wave; q < SN * SM; q += WAVES) {
      const int j = q / SM, m = q % SM;
      f32x4 s = s_part[turn][0][j][m][lane];
      for (int w = 1; w < WAVES; ++w) s += s_part[turn][w][j][m][lane];
      const int row = m0 + m * 16 + l16;
      if (row < n_rows)
        store4(p.C, F32, ((int64_t)lo + row) * p.N, n0 + j * 16 + 4 * kb, p.N, s);
    }
  }
}

// ------------------------------------------------------------ tiles in LDS
//
// 2 x WN waves, each TM x TN of a tile.  A slab is 128 deep: one scale group, 128
// bytes of each row of A and of B, so every global access is whole lines.  A ring of
// NST slabs in LDS is filled by hand-issued buffer_load ... lds (gemm_device.hpp);
// the loads of slab g + NST - 1 are spread over the MFMAs of a slab period, across
// tiles too.  A's scale bytes travel with their slab, each into a word of its own
// (rows of an expert start anywhere, so that wider loads would not be aligned); B's
// one byte per block of 128 columns is the same for a whole wave and comes through
// the scalar cache.
//
// Which rows make up an MFMA block is free: block b of a wave holds every SM-th
// (SN-th) row, from row b on, so that a lane reads the scale words of all its blocks
// at once and stores SN consecutive columns.  Which k an MFMA's lanes take is free
// too, as long as both operands agree and a scale covers them all.
//
// Measured: 8192^3 385 us (2.85 PFLOP/s), to fp32 765; 65536 rows of 64 experts x 4096 x
// 4096 1003 us.  Bound by the matrix cores (in use 0.65 of the time), the loads' arrival,
// the tiles that an expert's last rows leave part empty (there an eighth) and the stores
// (7% there).
template <int BM, int BN, int NST_, int WN_>
struct Shape {
  static constexpr int NST = NST_;
  static constexpr int WN = WN_, WAVES = 2 * WN;
  static constexpr int TM = BM / 2, TN = BN / WN;
  static constexpr int SM = TM / 32, SN = TN / 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, SA_BYTES = BM * 4;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES;
  static constexpr int SPARE = NST * STAGE;                // what waves without scales of their own load
  static constexpr int LDS_BYTES = SPARE + 256;            // and the experts' tables behind it
  static constexpr int NA = BM / 8 / WAVES, NB = BN / 8 / WAVES;  // 1 KB operand loads per wave per slab
  static constexpr int NL = NA + NB + 1;                   // + 64 scale bytes
  static constexpr int NMF = SM * SN;                      // MFMA blocks
  static_assert((SM == 2 || SM == 4) && (SN == 2 || SN == 4), "a row's scale words in one LDS read");
  static_assert(NA % 2 == 0 && NB % 2 == 0 && BM / 64 <= WAVES && TN <= 128, "whole loads per wave");
};

// LDS layout of an operand.  Block i of a wave's BLOCKS 32-row blocks is made of the
// rows l * BLOCKS + i (l = 0 .. 31) of the wave's part.  Eight consecutive rows, 128
// bytes each, are a 1 KB chunk; within it rows of one block stand together, and a
// row's 16-byte pieces are permuted by l >> 1.  So a ds_read_b128, served 16 lanes
// (16 consecutive l of one block and piece) at a time, meets all 16 slots of a
// 256-byte window.
template <int BLOCKS>
__device__ __forceinline__ int slot_row(int slot) {  // row of a slot of the chunk
  return BLOCKS == 4 ? 4 * (slot & 1) + (slot >> 1) : 2 * (slot & 3) + (slot >> 2);
}
template <int BLOCKS>
__device__ __forceinline__ int row_slot(int l) {  // bytes to row l of block 0 (block i: + i * 1024 / BLOCKS)
  return BLOCKS == 4 ? (l >> 1) * 1024 + (l & 1) * 128 : (l >> 2) * 1024 + (l & 3) * 128;
}
// The part of l >> 1 (mod 8) that the chunk's index gives.
template <int BLOCKS>
__device__ __forceinline__ constexpr unsigned piece_flip(int chunk) {
  return BLOCKS == 4 ? (unsigned)chunk & 7u : 2u * ((unsigned)chunk & 3u);
}

template <class F, int... I>
__device__ __forceinline__ void static_for_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_of(f, std::make_integer_sequence<int, N>{});
}

// W (2 or 4) columns at p, those before `left`; non-temporal where NT.
#define PGK_STORE(NT, type, p, ...)                                         \
  do {                                                                      \
    if constexpr (NT)                                                       \
      __builtin_nontemporal_store(__VA_ARGS__, reinterpret_cast<type*>(p)); \
    else                                                                    \
      *reinterpret_cast<type*>(p) = __VA_ARGS__;                            \
  } while (0)
template <int W, bool NT>
__device__ __forceinline__ void store_row(float* p, const float (&v)[W], int left) {
  if (left >= W) {
    if constexpr (W == 4)
      PGK_STORE(NT, u32x4_a4, p, __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
    else
      PGK_STORE(NT, u32x2_a4, p, __builtin_bit_cast(u32x2, f32x2{v[0], v[1]}));
  } else {
#pragma unroll
    for (int e = 0; e < W - 1; ++e)
      if (e < left) p[e] = v[e];
  }
}
template <int W, bool NT>
__device__ __forceinline__ void store_row(unsigned short* p, const float (&v)[W], int left) {
  unsigned o[W / 2];
#pragma unroll
  for (int e = 0; e < W / 2; ++e) o[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if (left >= W) {
    if constexpr (W == 4)
      PGK_STORE(NT, u32x2_a2, p, u32x2{o[0], o[1]});
    else
      PGK_STORE(NT, u32_a2, p, o[0]);
  } else {
#pragma unroll
    for (int e = 0; e < W - 1; ++e)
      if (e < left) p[e] = (unsigned short)(o[e >> 1] >> (16 * (e & 1)));
  }
}

constexpr int kGroupRows = 8;  // rows of tiles per group of an expert's grouped order

template <int BM, int BN, int NST, int WN, bool F32>
__global__ void __launch_bounds__(128 * WN) gemm_experts_tile_kernel(ExpertsParams p) {
  using S = Shape<BM, BN, NST, WN>;
  constexpr int NA = S::NA, NB = S::NB, NO = NA + NB, NL = S::NL, NMF = S::NMF;
  constexpr int SM = S::SM, SN = S::SN;
  // Of a period's 2 * NMF block positions the loads take the first SPREAD: half of
  // them where the ring's second stage has to have landed by the next period.
  constexpr int SPREAD = NST > 2 ? 2 * NMF : NMF;

  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  int* s_lo = reinterpret_cast<int*>(smem + S::LDS_BYTES);
  int* s_n = s_lo + p.experts;
  int* s_tile = s_n + p.experts;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, kb = lane >> 5;
  const int G = (int)gridDim.x;
  const int nk = p.K >> 7, nb = (p.N + 127) >> 7;
  const int npn = (p.N + BN - 1) / BN;

  expert_tiles(p.offsets, p.experts, p.rows, BM, npn, s_lo, s_n, s_tile);
  const int total = __builtin_amdgcn_readfirstlane(s_tile[p.experts]);

  // A tile: its expert, rows and columns.
  struct Tile {
    int t, e, lo, n, m0, n0;
  };
  auto open = [&](int t, Tile& x) {
    x.t = t;
    if (t >= total) return;
    x.e = __builtin_amdgcn_readfirstlane(expert_of_tile(s_tile, p.experts, t, x.e));
    x.lo = __builtin_amdgcn_readfirstlane(s_lo[x.e]);
    x.n = __builtin_amdgcn_readfirstlane(s_n[x.e]);
    const int npm = (x.n + BM - 1) / BM;
    int pm, pn;
    pgs::decode(pgs::kGrouped, t - __builtin_amdgcn_readfirstlane(s_tile[x.e]), npm, npn, kGroupRows, pm, pn);
    x.m0 = __builtin_amdgcn_readfirstlane(pm) * BM;
    x.n0 = __builtin_amdgcn_readfirstlane(pn) * BN;
  };

  // Global -> LDS.  Operands: instruction q covers rows 8q .. 8q + 7, lane i
  // slot i / 8 of LDS chunk q; instruction d of wave w is q = w * N + d.
  const int r8 = lane >> 3;
  const unsigned rowb = (unsigned)p.K;
  const unsigned aoff = (unsigned)(wave * NA * 8 + slot_row<SM>(r8)) * rowb;
  const unsigned boff = (unsigned)(wave * NB * 8 + slot_row<SN>(r8)) * rowb;
  // 16-byte piece of the lane in instruction 0, in bytes; d flips bits of it
  const unsigned apiece = ((unsigned)((lane & 7) ^ (SM == 2 ? r8 >> 1 & 1 : 0)) ^ piece_flip<SM>(wave * NA)) * 16u;
  const unsigned bpiece = ((unsigned)((lane & 7) ^ (SN == 2 ? r8 >> 1 & 1 : 0)) ^ piece_flip<SN>(wave * NB)) * 16u;
  const bool scales_here = wave < BM / 64;  // 64 rows' scales
  const unsigned lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // LDS reads: piece 2 q + kb of row l32 of a block; step h takes q = 2 h and 2 h + 1.
  unsigned rd_a[4], rd_b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const unsigned c = (unsigned)((2 * q + kb) ^ (l32 >> 1 & 7)) * 16u;
    rd_a[q] = (unsigned)(wm * S::TM * 128 + row_slot<SM>(l32)) + c;
    rd_b[q] = (unsigned)(S::A_BYTES + wn * S::TN * 128 + row_slot<SN>(l32)) + c;
  }
  const unsigned rd_sa = (unsigned)(S::A_BYTES + S::B_BYTES + (wm * S::TM + l32 * SM) * 4);

  // ---- loader ----
  Tile lt = {0, 0, 0, 0, 0, 0};
  int lk = 0;  // next slab
  rsrc_words_t rA, rB, rS;
  unsigned long long a_ptr = 0, b_ptr = 0, s_ptr = 0, sb_ptr = 0;
  unsigned a_rec = 0, b_rec = 0, s_rec = 0;
  unsigned sbw[NST - 1] = {}, sbs[NST - 1] = {};  // words with B's scale byte, of the slabs on their way, and its place

  auto begin_tile = [&](int t) {
    open(t, lt);
    lk = 0;
    if (t >= total) return;
    const int ra = lt.n - lt.m0 < BM ? lt.n - lt.m0 : BM, rb = p.N - lt.n0 < BN ? p.N - lt.n0 : BN;
    a_ptr = reinterpret_cast<unsigned long long>(p.A + ((int64_t)lt.lo + lt.m0) * p.K);
    b_ptr = reinterpret_cast<unsigned long long>(p.B + ((int64_t)lt.e * p.N + lt.n0) * p.K);
    a_rec = (unsigned)ra * rowb;
    b_rec = (unsigned)rb * rowb;
    const int sr = ra - wave * 64;
    s_ptr = reinterpret_cast<unsigned long long>(p.sa + lt.lo + lt.m0 + wave * 64);
    s_rec = scales_here && sr > 0 ? (unsigned)sr : 0u;
    const int blk = (lt.n0 >> 7) + wn * S::TN / 128;
    sb_ptr = reinterpret_cast<unsigned long long>(p.sb + ((int64_t)lt.e * nb + (blk < nb ? blk : nb - 1)) * nk);
  };
  // The next slab's resources; without one they are empty and the loads read
  // zeros into a stage no one reads.
  auto prep = [&]() {
    if (lt.t < total && lk == nk) begin_tile(lt.t + G);
    const bool load = lt.t < total;
    const unsigned k0 = (unsigned)lk * 128u;
    rA = rsrc_words_u64(a_ptr + k0, load ? a_rec - k0 : 0u);
    rB = rsrc_words_u64(b_ptr + k0, load ? b_rec - k0 : 0u);
    rS = rsrc_words_u64(s_ptr + (unsigned long long)lk * (unsigned long long)p.rows, load ? s_rec : 0u);
#pragma unroll
    for (int i = 0; i + 1 < NST - 1; ++i) {
      sbw[i] = sbw[i + 1];
      sbs[i] = sbs[i + 1];
    }
    if (load) {
      // the aligned word that holds the byte, which is taken out when the slab's turn
      // comes: a wait here would hold up the MFMAs
      const unsigned long long at = sb_ptr + (unsigned)lk;
      sbw[NST - 2] = *reinterpret_cast<const __attribute__((address_space(4))) unsigned*>(at & ~3ull);
      sbs[NST - 2] = 8u * ((unsigned)at & 3u);
      ++lk;
    }
  };
  auto dma = [&](int st, int d) PGK_INLINE {
    const unsigned sb = lds0 + (unsigned)(st * S::STAGE);
    if (d < NA) {
      load_lds16(rA, sb + (unsigned)((wave * NA + d) * 1024), aoff + (unsigned)d * 8u * rowb + (apiece ^ (piece_flip<SM>(d) * 16u)));
    } else if (d < NO) {
      const int e = d - NA;
      load_lds16(rB, sb + (unsigned)(S::A_BYTES + (wave * NB + e) * 1024),
                 boff + (unsigned)e * 8u * rowb + (bpiece ^ (piece_flip<SN>(e) * 16u)));
    } else {
      load_lds_u8(rS, scales_here ? sb + (unsigned)(S::A_BYTES + S::B_BYTES + wave * 256) : lds0 + (unsigned)S::SPARE,
                  (unsigned)lane);
    }
  };

  f32x16 acc[SN][SM];
  u32x4 aq[2][SM][2], bq[2][SN][2];  // fragments, by the step
  unsigned wa[2][SM];                // A's scale words, of the slab and the one before
  unsigned wb[2] = {};               // B's

  // LDS read r of step h: B block 0, the A blocks, the other B blocks (the order the
  // MFMAs consume them), two pieces each; step 0 the scale words first.
  constexpr int NR = 2 * (SM + SN);
  auto read = [&](int st, auto hc, int r) PGK_INLINE {
    constexpr int h = hc;
    const unsigned char* s = smem + st * S::STAGE;
    const int i = r >> 1, q = 2 * h + (r & 1);
    if (i == 0)
      bq[h][0][r & 1] = *reinterpret_cast<const u32x4*>(s + rd_b[q]);
    else if (i <= SM)
      aq[h][i - 1][r & 1] = *reinterpret_cast<const u32x4*>(s + rd_a[q] + (i - 1) * (1024 / SM));
    else
      bq[h][i - SM][r & 1] = *reinterpret_cast<const u32x4*>(s + rd_b[q] + (i - SM) * (1024 / SN));
  };
  auto read_scales = [&](int st, int par) PGK_INLINE {
    const unsigned* w = reinterpret_cast<const unsigned*>(smem + st * S::STAGE + rd_sa);
#pragma unroll
    for (int i = 0; i < SM; ++i) wa[par][i] = w[i];
  };
  auto mfma = [&](auto hc, auto jc, int par) PGK_INLINE {
    constexpr int h = hc, sn = jc / SM, sm = jc % SM;
    const u32x4 a0 = aq[h][sm][0], a1 = aq[h][sm][1], b0 = bq[h][sn][0], b1 = bq[h][sn][1];
    if constexpr (F32) {
      const Exact a(aq[h][sm], scale_value(wa[par][sm])), b(bq[h][sn], scale_value(wb[par]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[sn][sm] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v[i], b.v[i], acc[sn][sm], 0, 0, 0);
    } else {
      acc[sn][sm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          i32x8{(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]},
          i32x8{(int)b0[0], (int)b0[1], (int)b0[2], (int)b0[3], (int)b1[0], (int)b1[1], (int)b1[2], (int)b1[3]},
          acc[sn][sm], kFmtE4M3, kFmtE4M3, 0, (int)wa[par][sm], 0, (int)wb[par]);
    }
  };
  // Step h on the matrix cores (of a period that runs step 1 of the slab before,
  // then step 0); the next step's reads (of stage st_rd) and the loads that fall on
  // this half of the period.
  auto step = [&](auto hc, int par, int st_rd, int st_dma) PGK_INLINE {
    static_for<NMF>([&](auto jc) PGK_INLINE {
      constexpr int h = hc, j = jc, nx = 1 - h;
      mfma(hc, jc, par);
      static_for<NR>([&](auto rc) PGK_INLINE {
        if constexpr (rc * NMF / NR == j) read(st_rd, std::integral_constant<int, nx>{}, rc);
      });
      static_for<NL>([&](auto dc) PGK_INLINE {
        if constexpr (dc * SPREAD / NL == (1 - h) * NMF + j) dma(st_dma, dc);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Lane l holds SN consecutive columns, l % 32 * SN of the wave's, one per
  // block; registers 4 g + e hold rows (8 g + 4 (l / 32) + e) * SM + block: a
  // store of the wave covers two rows' 32 * SN consecutive columns.
  typedef std::conditional_t<F32, float, unsigned short> out_t;
  auto put_tile = [&](const Tile& x, auto edge, auto nt) {
    const int n = x.n0 + wn * S::TN + l32 * SN, m = x.m0 + wm * S::TM + 4 * kb * SM;
    out_t* base = static_cast<out_t*>(p.C) + ((int64_t)x.lo + m) * p.N + n;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < SM; ++i) {
          const int r = (8 * g + e) * SM + i;
          if (edge && m + r >= x.n) continue;
          float v[SN];
#pragma unroll
          for (int j = 0; j < SN; ++j) v[j] = acc_read(acc[j][i][4 * g + e]);
          store_row<SN, nt>(base + (int64_t)r * p.N, v, edge ? p.N - n : SN);
        }
  };
  // Whole tiles whose rows consist of whole lines are stored past the caches (us, past them
  // / through them, 16 experts x 4096 x 1024, bf16 C of 16 MB 16.6 / 17.9, 64 MB 42.2 / 43.3, 256
  // MB 152 / 188, fp32 256 MB 143 / 146; with the activation that reads C next, 27.4 / 28.0, 73.6 /
  // 75.2 and 250 / 275).
  auto epilogue = [&](const Tile& x) {
    const bool edge = x.m0 + BM > x.n || x.n0 + BN > p.N;
    const bool lines = (p.N & (F32 ? 31 : 63)) == 0 && (reinterpret_cast<uintptr_t>(p.C) & 127) == 0;
    const std::integral_constant<bool, true> yes;
    const std::integral_constant<bool, false> no;
    if (edge)
      put_tile(x, yes, no);
    else if (lines)
      put_tile(x, no, yes);
    else
      put_tile(x, no, no);
  };

  // programs of one XCD take consecutive tiles: they share operand panels in its L2
  const int first = pgs::program_of(blockIdx.x, G, p.xcds, 1);
  Tile ct = {0, 0, 0, 0, 0, 0};
  open(first, ct);
  if (first >= total) return;
  begin_tile(first);
#pragma unroll
  for (int j = 0; j < NST - 1; ++j) {
    prep();
#pragma unroll
    for (int d = 0; d < NL; ++d) dma(j, d);
  }
  // Slab g has landed once this wave's loads of it are done (those of the NST - 2
  // slabs after it may be in flight) and every wave has passed the barrier; every wave
  // has then finished its LDS reads of slab g - 1, which frees that stage for slab g +
  // NST - 1.
  int g = 0;
  const std::integral_constant<int, 0> step0;
  const std::integral_constant<int, 1> step1;
  auto slab_start = [&](int& st, int& st_dma) {
    wait_vm<(NST - 2) * NL>();
    slab_barrier();
    __builtin_amdgcn_sched_barrier(0);
    st = g % NST;
    st_dma = st == 0 ? NST - 1 : st - 1;
    wb[0] = wb[1];
    wb[1] = sbw[0] >> sbs[0] & 0xffu;
#pragma unroll
    for (int i = 0; i < SM; ++i) wa[0][i] = wa[1][i];
    ++g;
  };
  while (ct.t < total) {
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int i = 0; i < SM; ++i) acc[j][i] = f32x16{};
    int st, st_dma;
    slab_start(st, st_dma);
    read_scales(st, 1);
#pragma unroll
    for (int r = 0; r < NR; ++r) read(st, step0, r);
    __builtin_amdgcn_sched_barrier(0);
    prep();
#pragma unroll
    for (int d = 0; d < NL; ++d)
      if (d * SPREAD / NL < NMF) dma(st_dma, d);
    step(step0, 1, st, st_dma);
    for (int ck = 1; ck < nk; ++ck) {
      slab_start(st, st_dma);
      read_scales(st, 1);
      prep();
      __builtin_amdgcn_sched_barrier(0);
      step(step1, 0, st, st_dma);
      step(step0, 1, st, st_dma);
    }
    static_for<NMF>([&](auto jc) PGK_INLINE { mfma(step1, jc, 1); });
    mfma_results_ready();
    epilogue(ct);
    open(ct.t + G, ct);
  }
  // the loads of stages that no one reads have to land before the workgroup's LDS is
  // given away
  wait_vm<0>();
}

}  // namespace

namespace {

constexpr int kDevices = 64;
int tables_bytes(int experts) { return (3 * experts + 1) * (int)sizeof(int); }

// Resident workgroups per CU, asked for once per kernel and device (the answer, and
// the LDS limit it sets, cost microseconds of a short call); with the largest tables.
struct Instance {
  int bm, bn, threads, lds;
  void (*kern)(ExpertsParams);
  mutable std::atomic<int> resident[kDevices] = {};
  int per_cu() const {
    int dev = 0;
    const int most = lds + tables_bytes(kMaxExperts);
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices)
      return occupancy_of(reinterpret_cast<const void*>(kern), threads, most);
    int n = resident[dev].load(std::memory_order_acquire);
    if (n == 0) {
      n = occupancy_of(reinterpret_cast<const void*>(kern), threads, most);
      resident[dev].store(n, std::memory_order_release);
    }
    return n;
  }
};

template <int BM, int BN, int NST, int WN, bool F32>
Instance tiled() {
  return {BM, BN, 128 * WN, Shape<BM, BN, NST, WN>::LDS_BYTES, gemm_experts_tile_kernel<BM, BN, NST, WN, F32>};
}

}  // namespace

// The kernel and tile of a call, from its sizes alone (the experts' row counts are in
// device memory).  `few`: experts that can have rows.
//
// Streaming, for up to 12 rows per expert: rows of B at 6 TB/s (us, 4096 x 4096, 64
// experts, 32 / 64 columns a tile, against 128 x 128 tiles: 8 rows 28.5 / 24.8, 128
// rows 152 / 151 and more than 218, 512 rows 198 / 191 and 220, 1024 rows 282 / 243
// and 229; one matrix of 8192 x 8192, 1 row 15.5 / 20.4 and 32.5).  64 columns where
// their tiles give every CU one.  Up to 64 rows too where 128 x 128 tiles would leave
// half of the CUs idle, with tiles of 32 or 64 rows (8192 x 8192, 32 rows 19.6 against
// 33.7; 64 rows 29.2 against 35.5).
//
// Tiles: the least of the estimated times, rounds of tiles times what a CU needs for
// one, us for a 128-deep slab and for the rest (128 x 128 0.57 and 2, 128 x 256 0.83
// and 3, both on rings of three slabs; 256 x 256 1.45 and 8).  us measured, 128 x 128 /
// 128 x 256 / 256 x 256: 64 experts x 4096 x 4096, 4096 rows 245 / 247 / 281, 16384
// rows 421 / 350 / 380, 32768 rows 712 / 580 / 586; one of 8192 x 8192, 512 rows 39 / 56
// / 96, 1024 rows 77 / 59 / 96, 4096 rows 280 / 217 / 202.
hipError_t launch_gemm_experts(const ExpertsParams& p, int cus, hipStream_t stream) {
  const int tables = tables_bytes(p.experts), f32 = p.out_f32 ? 1 : 0;
  const int64_t few = p.rows < p.experts ? p.rows : p.experts;
  auto columns = [&](int bn) { return (int64_t)(p.N + bn - 1) / bn; };
  if (p.rows <= 12LL * p.experts || (p.rows <= 64LL * p.experts && 2 * few * columns(128) <= cus)) {
    typedef void (*kern_t)(ExpertsParams);
    static const kern_t all[4][2] = {
        {gemm_experts_stream_kernel<1, 2, 4, 4, false>, gemm_experts_stream_kernel<1, 2, 4, 4, true>},
        {gemm_experts_stream_kernel<1, 4, 2, 4, false>, gemm_experts_stream_kernel<1, 4, 2, 4, true>},
        {gemm_experts_stream_kernel<2, 2, 2, 4, false>, gemm_experts_stream_kernel<2, 2, 2, 4, true>},
        {gemm_experts_stream_kernel<4, 2, 2, 4, false>, gemm_experts_stream_kernel<4, 2, 2, 4, true>}};
    const int i = p.rows > 32LL * p.experts ? 3 : p.rows > 16LL * p.experts ? 2 : few * columns(64) >= cus ? 1 : 0;
    hipLaunchKernelGGL(all[i][f32], dim3(4 * cus), dim3(256), tables, stream, p);
    return hipGetLastError();
  }
  static const Instance all[3][2] = {{tiled<128, 128, 3, 2, false>(), tiled<128, 128, 3, 2, true>()},
                                     {tiled<128, 256, 3, 2, false>(), tiled<128, 256, 3, 2, true>()},
                                     {tiled<256, 256, 2, 2, false>(), tiled<256, 256, 2, 2, true>()}};
  static const double cost[3][2] = {{0.57, 2}, {0.83, 3}, {1.45, 8}};
  int best = 0;
  double least = 0;
  for (int i = 0; i < 3; ++i) {
    const Instance& x = all[i][0];
    // an expert's last tile is half full, but has one tile at least
    int64_t row_tiles = p.experts == 1 ? (p.rows + x.bm - 1) / x.bm : p.rows / x.bm + p.experts / 2;
    if (row_tiles < few) row_tiles = few;
    const int64_t rounds = (row_tiles * columns(x.bn) + cus - 1) / cus;
    const double us = (double)rounds * (cost[i][0] * (p.K >> 7) + cost[i][1]);
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  const Instance& x = all[best][f32];
  hipLaunchKernelGGL(x.kern, dim3(cus * x.per_cu()), dim3(x.threads), x.lds + tables, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
