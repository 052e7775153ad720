// Persistent MXFP4 GEMM for gfx950: C[M][N] = A . B^T with A[M][K] and
// B[N][K] OCP e2m1 codes (two to a byte) and one e8m0 scale byte per 32
// consecutive k (SA[K/128][M][4], SB[K/128][N][4]), fp32 accumulate, C bf16
// or fp32.
//
// Two kernels:
//  * gemm_fp4_kernel, tiles staged through LDS, on v_mfma_scale_f32_32x32x64:
//    bound by how fast a CU's loads arrive (8192^3 237 to 257 us, 4.3 to 4.6
//    PFLOP/s, the first fifty calls of a run the slowest; 172 to 184 us with the
//    loads taken out).
//  * gemm_fp4_skinny_kernel for few rows, on v_mfma_scale_f32_16x16x128: bound by
//    the bytes of B (1 x 28672 x 8192 26 to 32 us, 3.9 to 4.75 TB/s), which each wave streams
//    straight into registers; the waves of a workgroup split K and add their
//    sums in LDS.
// In both, a lane supplies the 32 k-values of one row and block as 16 bytes
// and the scale byte of exactly that block.
#include <atomic>
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "gemm_device.hpp"

namespace pgk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFmtE2M1 = 4;  // f8f6f4 operand format code of e2m1
constexpr int kMaxWaves = 8;  // of a workgroup of the kernel for few rows
constexpr int BK = 256;      // k per slab: 128 bytes of a row, two scale groups

// f(0) .. f(N - 1) with compile-time arguments (the MFMA's opsel and the
// places of loads among the MFMAs are immediates).
template <class F, int... I>
__device__ __forceinline__ void static_for_of(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_of(f, std::make_integer_sequence<int, N>{});
}
#define PGK_INLINE __attribute__((always_inline))

template <int OPSEL_A, int OPSEL_B>
__device__ __forceinline__ f32x4 mfma_scaled(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                          i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, kFmtE2M1,
                                                          kFmtE2M1, OPSEL_A, sa, OPSEL_B, sb);
}

template <int OPSEL_A, int OPSEL_B>
__device__ __forceinline__ f32x16 mfma_scaled32(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                         i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, kFmtE2M1,
                                                         kFmtE2M1, OPSEL_A, sa, OPSEL_B, sb);
}

// Rows of C start on any element; stores of any alignment are single
// instructions.  Columns c .. c + 3 of a row of C that ends at n:
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef unsigned u32_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void store_f32x4(float* row, int64_t c, int64_t n, f32x4 v) {
  if (c + 4 <= n) {
    *reinterpret_cast<u32x4_a4*>(row + c) = __builtin_bit_cast(u32x4, v);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (c + e < n) row[c + e] = v[e];
  }
}
// W (2 or 4) columns at p, those before `left`; non-temporal where NT.
// (Macro: a template would drop the alignment of the typedefs above.)
#define PGK_STORE(NT, type, p, ...)                                               \
  do {                                                                            \
    if constexpr (NT)                                                             \
      __builtin_nontemporal_store(__VA_ARGS__, reinterpret_cast<type*>(p));       \
    else                                                                          \
      *reinterpret_cast<type*>(p) = __VA_ARGS__;                                  \
  } while (0)
template <int W, bool NT>
__device__ __forceinline__ void store_row(float* p, const float (&v)[W], int64_t left) {
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
__device__ __forceinline__ void store_row(unsigned short* p, const float (&v)[W], int64_t left) {
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

// ------------------------------------------------------------ tiles in LDS
//
// 2 x WN waves, each TM x TN of the tile.  A slab is 256 deep: 128 bytes of
// each row of A and of B, so every global access is whole 128-byte lines (64-byte
// pieces of twice the rows: 8192^3 290 -> 326 us), and the scale words of its
// two 128-deep groups.  A ring of NST slabs in LDS is filled by hand-issued
// buffer_load ... lds (gemm_device.hpp); the loads of slab g + NST - 1 are
// spread over the MFMAs of a slab period, across tiles too.  What a load costs
// is its instruction more than its bytes (8192^3 at four waves: 184 us with
// none, 204 with the scales' alone, 270 with the operands', 290 with both), so
// all are 16 bytes a lane.  At 256 x 256, eight waves are level with four on
// long K and gain 6% where K is short (3000 x 7000 x 2048 46 -> 43 us): two waves
// on a SIMD cover each other's barriers and stores.
//
// Which rows make up an MFMA block is free, and chosen so that a lane's scale
// words and its results are consecutive: block b of a wave holds every SM-th
// (SN-th) row, from row b on.  A lane then reads the words of all its blocks
// with one ds_read_b128 (b64 for two blocks) from words that came in memory
// order, gathers its own byte of each into one register (v_perm), from which
// the MFMA selects by opsel, and stores SN consecutive columns, 32 lanes a
// stretch of 32 * SN of a row of C.  (Blocks of consecutive rows, words loaded
// four bytes a lane to reorder them: 8192^3 274 us, 256 x 28672 x 8192 55 against
// 260 and 47.)
template <int BM, int BN, int NST_, int WN_>
struct Shape {
  static constexpr int NST = NST_;
  static constexpr int WN = WN_, WAVES = 2 * WN;  // 2 x WN waves
  static constexpr int TM = BM / 2, TN = BN / WN;
  static constexpr int SM = TM / 32, SN = TN / 32;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SA_BYTES = BM * 8, SB_BYTES = BN * 8;  // two groups of words
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int LDS_BYTES = NST * STAGE + 16 + (WAVES > 4 ? 1024 : 0);  // + first tile, next tile [2]
  static constexpr int NA = BM / 8 / WAVES, NB = BN / 8 / WAVES;  // 1 KB operand loads per wave per slab
  static constexpr int NL = NA + NB + 1;              // + one 1 KB load of scale words
  static constexpr int NMF = SM * SN;                 // MFMAs per 64-deep step
  static_assert((SM == 2 || SM == 4) && (SN == 2 || SN == 4), "a row's scale words in one LDS read");
  static_assert(BM % 128 == 0 && BN % 128 == 0 && NA % 2 == 0 && NB % 2 == 0, "whole loads per wave");
};

// LDS layout of an operand.  Block i of a wave's BLOCKS 32-row blocks is made
// of the rows l * BLOCKS + i (l = 0 .. 31) of the wave's half.  Eight
// consecutive rows, 128 bytes each, are a 1 KB chunk; within it rows of one
// block stand together, and a row's 16-byte pieces are permuted by l >> 1.
// So a ds_read_b128, served 16 lanes (16 consecutive l of one block and
// piece) at a time, meets all 16 slots of a 256-byte window.
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

// The scale words of one row of each of the wave's blocks.
template <int BLOCKS>
struct Words {
  typedef u32x4 type;
};
template <>
struct Words<2> {
  typedef u32x2 type;
};

template <int BM, int BN, int NST, int WN, bool GRP>
__global__ void __launch_bounds__(128 * WN) gemm_fp4_kernel(GemmParams P) {
  using S = Shape<BM, BN, NST, WN>;
  constexpr int NA = S::NA, NB = S::NB, NO = NA + NB, NL = S::NL, NMF = S::NMF;
  constexpr int SM = S::SM, SN = S::SN;
  // Of a period's 4 * NMF MFMA positions, the loads take the first SPREAD: half
  // of them where the ring's second stage has to have landed by the next period.
  constexpr int SPREAD = NST > 2 ? 4 * NMF : 2 * NMF;

  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  int* s_first = reinterpret_cast<int*>(smem + NST * S::STAGE);
  int* s_next = s_first + 1;  // [2]: the loader's next tile, by claim parity

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, kb = lane >> 5;
  const int prog = pgs::program_of(blockIdx.x, P.s.G, P.s.X, P.s.xcd_major);
  // the loader tile's problem and the matrix cores' tile's problem
  int Ml = P.M, Nl = P.N, Kl = P.K;
  const unsigned char* Al = static_cast<const unsigned char*>(P.A);
  const unsigned char* Bl = static_cast<const unsigned char*>(P.B);
  const uint8_t* SAl = P.sa;
  const uint8_t* SBl = P.sb;
  int Mc = P.M, Nc = P.N;
  void* Cc = P.C;

  Walker walker(P.s, prog);
  const bool witness = P.w.visits != nullptr;
  if (witness) walker.claim_row = P.w.claims + (size_t)prog * kMaxStealCounters;
  long long t_start = 0, c_start = 0;
  if (witness && tid == 0) {
    t_start = wall_ticks();
    c_start = shader_cycles();
  }

  // Global -> LDS.  Operands: instruction q covers rows 8q .. 8q + 7, lane p
  // slot p / 8 of LDS chunk q; instruction d of wave w is q = w * N + d.
  const int r8 = lane >> 3;
  unsigned aoff = 0, boff = 0;  // row of instruction 0
  unsigned rowb = 0;
  auto lane_offsets = [&](int Kx) {
    rowb = (unsigned)Kx >> 1;
    aoff = (unsigned)(wave * NA * 8 + slot_row<SM>(r8)) * rowb;
    boff = (unsigned)(wave * NB * 8 + slot_row<SN>(r8)) * rowb;
  };
  lane_offsets(Kl);
  // 16-byte piece of the lane in instruction 0, in bytes; d flips bits of it
  const unsigned apiece = ((unsigned)((lane & 7) ^ (SM == 2 ? r8 >> 1 & 1 : 0)) ^ piece_flip<SM>(wave * NA)) * 16u;
  const unsigned bpiece = ((unsigned)((lane & 7) ^ (SN == 2 ? r8 >> 1 & 1 : 0)) ^ piece_flip<SN>(wave * NB)) * 16u;
  // Scale words, four rows of one group per lane: waves 0 and 1 A's, 2 and 3
  // B's; waves past them, which issue the same instruction, nothing, into a
  // kilobyte of their own.  256 rows: a group each; 128 rows: both groups, twice the same.
  const bool of_a = wave < 2;
  const int srows = of_a ? BM : BN;
  const int sgrp = srows == 256 ? (wave & 1) : (lane >> 5);
  const int srow = (srows == 256 ? lane : (lane & 31)) * 4;
  const unsigned slds = wave >= 4 ? (unsigned)(NST * S::STAGE + 16)
                                  : (unsigned)(S::A_BYTES + S::B_BYTES + (of_a ? 0 : S::SA_BYTES) +
                                               (srows == 256 ? (wave & 1) * 1024 : 0));
  const unsigned lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // LDS reads: step h: piece 2 h + kb of row l32 of a block.
  unsigned rd_a[4], rd_b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const unsigned c = (unsigned)((2 * q + kb) ^ (l32 >> 1 & 7)) * 16u;
    rd_a[q] = (unsigned)(wm * S::TM * 128 + row_slot<SM>(l32)) + c;
    rd_b[q] = (unsigned)(S::A_BYTES + wn * S::TN * 128 + row_slot<SN>(l32)) + c;
  }
  const unsigned rd_sa = (unsigned)(S::A_BYTES + S::B_BYTES + (wm * S::TM + l32 * SM) * 4);
  const unsigned rd_sb = (unsigned)(S::A_BYTES + S::B_BYTES + S::SA_BYTES + (wn * S::TN + l32 * SN) * 4);
  // v_perm selectors: byte kb (odd steps: kb + 2) of two words into the low or
  // the high half
  const unsigned sel_lo = 0x0c0c0400u + 0x0101u * (unsigned)kb;
  const unsigned sel_hi = 0x04000c0cu + 0x01010000u * (unsigned)kb;

  auto problem_of = [&](int v) {
    GemmProblem pr = P.gp[0];
#pragma unroll
    for (int q = 1; q < kMaxGemmProblems; ++q)
      if (q < P.ngemm && v >= P.gp[q].tile0) pr = P.gp[q];
    return pr;
  };
  auto coords = [&](int v, int& m0, int& n0) {
    int pm, pn;
    if (GRP) {
      const GemmProblem pr = problem_of(v);
      pgs::decode(P.s.kind, v - pr.tile0, pr.npm, pr.npn, P.s.gs, pm, pn);
    } else {
      walker.tile_coords(v, pm, pn);
    }
    m0 = pm * BM;
    n0 = pn * BN;
  };

  // ---- loader state ----
  int nkl = (Kl + BK - 1) / BK;  // slabs of the loader's tile
  int lt = -1, lk = 0;           // tile, next slab
  // tiles the loader moved on to that the matrix cores have not reached
  int pend[NST - 1];
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) pend[i] = -1;
  int claims = 0;
  int lm0 = 0, ln0 = 0;
  rsrc_words_t rA, rB, rS;
  unsigned long long a_ptr = 0, b_ptr = 0;
  unsigned a_rec = 0, b_rec = 0;
  unsigned ahalf = 0, bhalf = 0, hflip = 0;  // kOob in lanes whose piece is past K (instruction 0; flipped)
  unsigned soff = 0;

  auto begin_tile = [&](int t) {
    lt = t;
    lk = 0;
    if (GRP) {
      const GemmProblem pr = problem_of(t);
      Al = static_cast<const unsigned char*>(pr.A);
      Bl = static_cast<const unsigned char*>(pr.B);
      SAl = pr.sa;
      SBl = pr.sb;
      Ml = pr.M;
      Nl = pr.N;
      Kl = pr.K;
      nkl = (Kl + BK - 1) / BK;
      lane_offsets(Kl);
    }
    coords(t, lm0, ln0);
    int ra = Ml - lm0 < BM ? Ml - lm0 : BM, rb = Nl - ln0 < BN ? Nl - ln0 : BN;
    ra = ra < 0 ? 0 : ra;
    rb = rb < 0 ? 0 : rb;
    const int rowb = Kl >> 1;
    a_ptr = reinterpret_cast<unsigned long long>(Al + (size_t)lm0 * rowb);
    b_ptr = reinterpret_cast<unsigned long long>(Bl + (size_t)ln0 * rowb);
    a_rec = (unsigned)(ra * rowb);
    b_rec = (unsigned)(rb * rowb);
    const int sm = of_a ? Ml : Nl, s0 = of_a ? lm0 : ln0;
    soff = wave < 4 && s0 + srow < sm ? (unsigned)(sgrp * sm + srow) * 4u : kOob;
  };

  // The next slab's resources; without one they are empty and the loads read
  // zeros into a stage no one reads.
  auto prep = [&]() {
    lt = __builtin_amdgcn_readfirstlane(lt);
    lk = __builtin_amdgcn_readfirstlane(lk);
    claims = __builtin_amdgcn_readfirstlane(claims);
    if (lt >= 0 && lk == nkl) {
      lt = -1;
      const int t = __builtin_amdgcn_readfirstlane(s_next[claims & 1]);
      ++claims;
      if (t >= 0) {
        bool queued = false;
#pragma unroll
        for (int i = 0; i < NST - 1; ++i)
          if (!queued && pend[i] < 0) {
            pend[i] = t;
            queued = true;
          }
        begin_tile(t);
      }
    }
    const int k0 = lk * BK;
    const bool load = lt >= 0;
    if (load) {
      ++lk;
      if (lk == nkl && tid == 0) s_next[claims & 1] = walker.next(lt);
    }
    rA = rsrc_words_u64(a_ptr + (unsigned long long)(k0 >> 1), load ? a_rec - (unsigned)(k0 >> 1) : 0u);
    rB = rsrc_words_u64(b_ptr + (unsigned long long)(k0 >> 1), load ? b_rec - (unsigned)(k0 >> 1) : 0u);
    // the second half of an odd last slab is past K: its pieces are past
    // every range, its scale words (the other group's rows) likewise
    const bool odd = k0 + 128 >= Kl;
    hflip = odd ? kOob : 0u;
    ahalf = (apiece & 64u) ? hflip : 0u;
    bhalf = (bpiece & 64u) ? hflip : 0u;
    const int grp = k0 >> 7, ng = odd ? 1 : 2;
    const int sm = of_a ? Ml : Nl, s0 = of_a ? lm0 : ln0;
    rS = rsrc_words_u64(reinterpret_cast<unsigned long long>((of_a ? SAl : SBl) + ((size_t)grp * sm + s0) * 4),
                        load ? (unsigned)(ng * sm - s0) * 4u : 0u);
  };

  auto dma = [&](int st, int d) PGK_INLINE {
    const unsigned sb = lds0 + (unsigned)(st * S::STAGE);
    if (d < NA) {
      const unsigned flip = piece_flip<SM>(d) * 16u;
      load_lds16(rA, sb + (unsigned)((wave * NA + d) * 1024),
                 (aoff + (unsigned)d * 8u * rowb + (apiece ^ flip)) | ((flip & 64u) ? ahalf ^ hflip : ahalf));
    } else if (d < NO) {
      const int e = d - NA;
      const unsigned flip = piece_flip<SN>(e) * 16u;
      load_lds16(rB, sb + (unsigned)(S::A_BYTES + (wave * NB + e) * 1024),
                 (boff + (unsigned)e * 8u * rowb + (bpiece ^ flip)) | ((flip & 64u) ? bhalf ^ hflip : bhalf));
    } else {
      load_lds16(rS, (wave < 4 ? sb : lds0) + slds, soff);
    }
  };

  f32x16 acc[SN][SM];
  i32x4 aq[2][SM], bq[2][SN];  // fragments, by the step's parity
  typedef typename Words<SM>::type wa_t;
  typedef typename Words<SN>::type wb_t;
  wa_t wa;  // scale words of a group: two steps
  wb_t wb;
  int sa = 0, sb = 0;  // gathered scale bytes of the step on the matrix cores

  // LDS read r of step h: B block 0, the A blocks, the other B blocks (the
  // order the MFMAs consume them); even steps the scale words too.
  auto reads = [](int h) { return SM + SN + (h % 2 == 0 ? 2 : 0); };
  auto read = [&](int st, int h, int r) PGK_INLINE {
    const unsigned char* p = smem + st * S::STAGE;
    if (r == 0)
      bq[h & 1][0] = *reinterpret_cast<const i32x4*>(p + rd_b[h]);
    else if (r <= SM)
      aq[h & 1][r - 1] = *reinterpret_cast<const i32x4*>(p + rd_a[h] + (r - 1) * (1024 / SM));
    else if (r < SM + SN)
      bq[h & 1][r - SM] = *reinterpret_cast<const i32x4*>(p + rd_b[h] + (r - SM) * (1024 / SN));
    else if (r == SM + SN)
      wa = *reinterpret_cast<const wa_t*>(p + rd_sa + (h >> 1) * BM * 4);
    else
      wb = *reinterpret_cast<const wb_t*>(p + rd_sb + (h >> 1) * BN * 4);
  };
  // byte kb + 2 u of each word (one per block)
  auto gather = [&](auto w, int u) {
    const unsigned d = 0x0202u * (unsigned)u;
    unsigned o = __builtin_amdgcn_perm(w[1], w[0], sel_lo + d);
    if constexpr (sizeof(w) == 16) o |= __builtin_amdgcn_perm(w[3], w[2], sel_hi + (d << 16));
    return (int)o;
  };
  auto scales = [&](int h) {
    sa = gather(wa, h & 1);
    sb = gather(wb, h & 1);
  };
  auto mfma = [&](auto hc, auto jc) PGK_INLINE {
    constexpr int b = hc & 1, sn = jc / SM, sm = jc % SM;
    acc[sn][sm] = mfma_scaled32<sm, sn>(aq[b][sm], bq[b][sn], acc[sn][sm], sa, sb);
  };
  // Step h on the matrix cores (of a period that runs steps 3, 0, 1, 2); the
  // next step's reads (of stage st_rd) and the loads that fall on this quarter
  // of the period.
  auto step = [&](auto hc, int st_rd, int st_dma) PGK_INLINE {
    scales(hc);
    __builtin_amdgcn_sched_barrier(0);
    static_for<NMF>([&](auto jc) PGK_INLINE {
      constexpr int h = hc, j = jc, nx = (h + 1) % 4, nr = SM + SN + (nx % 2 == 0 ? 2 : 0);
      mfma(hc, jc);
      static_for<nr>([&](auto rc) PGK_INLINE {
        if constexpr (rc * NMF / nr == j) read(st_rd, nx, rc);
      });
      static_for<NL>([&](auto dc) PGK_INLINE {
        if constexpr (dc * SPREAD / NL == nx * NMF + j) dma(st_dma, dc);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Lane l holds SN consecutive columns, l % 32 * SN of the wave's, one per
  // block; registers 4 g + e hold rows (8 g + 4 (l / 32) + e) * SM + block: a
  // store of the wave covers two rows' 32 * SN consecutive columns.
  auto put_tile = [&](int m0, int n0, auto out, auto edge, auto nt) {
    typedef decltype(out) T;
    const int64_t n = n0 + wn * S::TN + l32 * SN;
    const int m = m0 + wm * S::TM + 4 * kb * SM;
    T* base = static_cast<T*>(Cc) + (int64_t)m * Nc + n;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < SM; ++i) {
          const int r = (8 * g + e) * SM + i;
          if (edge && m + r >= Mc) continue;
          float v[SN];
#pragma unroll
          for (int j = 0; j < SN; ++j) v[j] = acc_read(acc[j][i][4 * g + e]);
          store_row<SN, nt>(base + (int64_t)r * Nc, v, edge ? (int64_t)Nc - n : (int64_t)SN);
        }
  };
  // Non-temporal where rows of C start on 128-byte lines, so that C does not
  // push operand panels out of L2 (8192^3 260 -> 250 us, 2000 x 28672 x 512 to
  // fp32 58 -> 51; 2048 x 4096 x 2048 18.3 -> 17.2, 1024 x 2048 x 1024 9.0 -> 8.7;
  // partial lines cost more than that: 3000 x 7000 x 2048 to fp32 44 against 48).
  // With a norm of C that follows at once, 4096 x 4096 x 4096 63.3 -> 65.8 us together
  // and 8192^3 338 -> 331.
  auto epilogue = [&](int m0, int n0) {
    const bool edge = m0 + BM > Mc || n0 + BN > Nc;
    const bool lines = (Nc & (P.out_f32 ? 31 : 63)) == 0 && (reinterpret_cast<uintptr_t>(Cc) & 127) == 0;
    const std::integral_constant<bool, true> yes;
    const std::integral_constant<bool, false> no;
    auto put = [&](auto out) {
      if (edge)
        put_tile(m0, n0, out, yes, no);
      else if (lines)
        put_tile(m0, n0, out, no, yes);
      else
        put_tile(m0, n0, out, no, no);
    };
    if (P.out_f32)
      put(0.0f);
    else
      put((unsigned short)0);
  };

  if (tid == 0) s_first[0] = walker.first();
  __syncthreads();
  int ct = __builtin_amdgcn_readfirstlane(s_first[0]);
  if (ct >= 0) {
    begin_tile(ct);
#pragma unroll
    for (int j = 0; j < NST - 1; ++j) {
      if (j > 0) slab_barrier();
      prep();
#pragma unroll
      for (int d = 0; d < NL; ++d) dma(j, d);
    }
  }
  int g = 0, it = 0, m0 = 0, n0 = 0;
  int cnk = (P.K + BK - 1) / BK;
  auto compute_tile = [&]() {
    coords(ct, m0, n0);
    if (GRP) {
      const GemmProblem pr = problem_of(ct);
      Mc = pr.M;
      Nc = pr.N;
      Cc = pr.C;
      cnk = (pr.K + BK - 1) / BK;
    }
  };
  if (ct >= 0) compute_tile();
  // Slab g has landed once this wave's loads of it are done (those of the NST
  // - 2 slabs after it may be in flight) and every wave has passed the
  // barrier; every wave has then finished its LDS reads of slab g - 1, which
  // frees that stage for slab g + NST - 1.
  auto slab_start = [&]() {
    wait_vm<(NST - 2) * NL>();
    slab_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<int, 0> step0;
  const std::integral_constant<int, 1> step1;
  const std::integral_constant<int, 2> step2;
  const std::integral_constant<int, 3> step3;
  while (ct >= 0) {
    if (tid == 0) {
      if (witness) {
        atomicAdd(P.w.visits + ct, 1);
        P.w.owner[ct] = prog;
        P.w.order[ct] = it;
      }
      if (is_straggler(P.s, prog)) spin_ns(P.s.straggler_ns, P.s.wall_khz);
    }
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int i = 0; i < SM; ++i) acc[j][i] = f32x16{};
    // A period per slab: the barrier, step 3 of the slab before (fragments in
    // registers) while step 0 of this one is read, then steps 0 to 2, each
    // while the next is read.  The tile's first slab has no step before it.
    {
      slab_start();
      const int st = g % NST, st_dma = st == 0 ? NST - 1 : st - 1;
#pragma unroll
      for (int r = 0; r < reads(0); ++r) read(st, 0, r);
      __builtin_amdgcn_sched_barrier(0);
      prep();
#pragma unroll
      for (int d = 0; d < NL; ++d)
        if (d * SPREAD / NL < NMF) dma(st_dma, d);
      step(step0, st, st_dma);
      step(step1, st, st_dma);
      step(step2, st, st_dma);
      ++g;
    }
    for (int ck = 1; ck < cnk; ++ck) {
      slab_start();
      const int st = g % NST, st_dma = st == 0 ? NST - 1 : st - 1;
      prep();
      __builtin_amdgcn_sched_barrier(0);
      step(step3, st, st_dma);
      step(step0, st, st_dma);
      step(step1, st, st_dma);
      step(step2, st, st_dma);
      ++g;
    }
    scales(3);
    static_for<NMF>([&](auto jc) PGK_INLINE { mfma(step3, jc); });
    mfma_results_ready();
    epilogue(m0, n0);
    ++it;
    ct = pend[0];
#pragma unroll
    for (int i = 0; i + 1 < NST - 1; ++i) pend[i] = pend[i + 1];
    pend[NST - 2] = -1;
    if (ct >= 0) compute_tile();
  }

  if (witness && tid == 0) {
    P.w.t_start[prog] = t_start;
    P.w.t_end[prog] = wall_ticks();
    P.w.cycles[prog] = shader_cycles() - c_start;
    P.w.hw_id[prog] = hw_placement();
    P.w.n_tiles[prog] = it;
  }
}

// ------------------------------------------------------------- a few rows
//
// A tile is 16 * SM rows by 16 * SN columns; each wave of the workgroup takes
// a stretch of K in units of 256 (per B row 128 bytes, one line, as two
// 16-byte loads per lane), DEPTH units in flight.  A comes from the caches.
// The waves' sums meet in LDS.
template <int SM, int SN, int DEPTH, bool GRP>
__global__ void __launch_bounds__(kMaxWaves * 64) gemm_fp4_skinny_kernel(GemmParams P) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  f32x4* s_part = reinterpret_cast<f32x4*>(smem);  // [2][waves][SN][SM][64], by the tile's parity
  __shared__ int s_tile[2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int l16 = lane & 15, kb = lane >> 4;
  const int prog = pgs::program_of(blockIdx.x, P.s.G, P.s.X, P.s.xcd_major);
  Walker walker(P.s, prog);
  const bool witness = P.w.visits != nullptr;
  if (witness) walker.claim_row = P.w.claims + (size_t)prog * kMaxStealCounters;
  long long t_start = 0, c_start = 0;
  if (witness && tid == 0) {
    t_start = wall_ticks();
    c_start = shader_cycles();
  }
  struct Tile {
    void* C;
    int M, N, m0, n0;
    const uint8_t *A, *B, *sa, *sb;
    int rowb, steps, ra, rb, u0, u1;
  };
  auto open = [&](int v, Tile& t) {
    GemmProblem pr;
    int pm, pn;
    if (GRP) {
      pr = P.gp[0];
#pragma unroll
      for (int q = 1; q < kMaxGemmProblems; ++q)
        if (q < P.ngemm && v >= P.gp[q].tile0) pr = P.gp[q];
      pgs::decode(P.s.kind, v - pr.tile0, pr.npm, pr.npn, P.s.gs, pm, pn);
    } else {
      pr.A = P.A;
      pr.B = P.B;
      pr.C = P.C;
      pr.sa = P.sa;
      pr.sb = P.sb;
      pr.M = P.M;
      pr.N = P.N;
      pr.K = P.K;
      walker.tile_coords(v, pm, pn);
    }
    t.C = pr.C;
    t.M = pr.M;
    t.N = pr.N;
    t.m0 = pm * 16 * SM;
    t.n0 = pn * 16 * SN;
    t.rowb = pr.K >> 1;
    t.steps = pr.K >> 7;
    t.ra = pr.M - t.m0 < 16 * SM ? pr.M - t.m0 : 16 * SM;
    t.rb = pr.N - t.n0 < 16 * SN ? pr.N - t.n0 : 16 * SN;
    t.A = static_cast<const uint8_t*>(pr.A) + (size_t)t.m0 * t.rowb;
    t.B = static_cast<const uint8_t*>(pr.B) + (size_t)t.n0 * t.rowb;
    t.sa = pr.sa + (size_t)t.m0 * 4;
    t.sb = pr.sb + (size_t)t.n0 * 4;
    // the wave's units: a consecutive stretch, so that a row's lines are read
    // one after the other
    const int units = (t.steps + 1) >> 1;
    t.u0 = units * wave / waves;
    t.u1 = units * (wave + 1) / waves;
  };
  struct Unit {
    u32x4 b[2][SN], a[2][SM];
    unsigned sb[2][SN], sa[2][SM];
  };
  // Unit u of a tile; rows past the operands read as zeros (range checks).
  auto load = [&](const Tile& t, int u, Unit& x) PGK_INLINE {
    const auto rA = rsrc(t.A, (unsigned)(t.ra * t.rowb));
    const auto rB = rsrc(t.B, (unsigned)(t.rb * t.rowb));
    const unsigned off = (unsigned)l16 * (unsigned)t.rowb + (unsigned)kb * 16u;
    const unsigned soff = (unsigned)(l16 * 4 + kb);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int st = u * 2 + s;
      const bool in = st < t.steps;  // uniform
      const unsigned at = in ? off + (unsigned)st * 64u : kOob;
      const auto rSA = rsrc(t.sa + (size_t)(in ? st : 0) * t.M * 4, (unsigned)(t.ra * 4));
      const auto rSB = rsrc(t.sb + (size_t)(in ? st : 0) * t.N * 4, (unsigned)(t.rb * 4));
#pragma unroll
      for (int j = 0; j < SN; ++j) {
        x.b[s][j] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, at + (unsigned)(j * 16) * (unsigned)t.rowb, 0, 0));
        x.sb[s][j] = __builtin_amdgcn_raw_buffer_load_b8(rSB, soff + j * 64, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < SM; ++i) {
        x.a[s][i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, at + (unsigned)(i * 16) * (unsigned)t.rowb, 0, 0));
        x.sa[s][i] = __builtin_amdgcn_raw_buffer_load_b8(rSA, soff + i * 64, 0, 0);
      }
    }
  };
  Tile t;
  Unit x[DEPTH];
  auto begin = [&](int v) PGK_INLINE {
    open(v, t);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (t.u0 + d < t.u1) load(t, t.u0 + d, x[d]);
  };
  if (tid == 0) s_tile[0] = walker.first();
  __syncthreads();
  int v = __builtin_amdgcn_readfirstlane(s_tile[0]);
  if (v >= 0) begin(v);
  int it = 0;
  while (v >= 0) {
    const int par = it & 1;
    if (tid == 0) {
      s_tile[par ^ 1] = walker.next(v);
      if (witness) {
        atomicAdd(P.w.visits + v, 1);
        P.w.owner[v] = prog;
        P.w.order[v] = it;
      }
      if (is_straggler(P.s, prog)) spin_ns(P.s.straggler_ns, P.s.wall_khz);
    }
    f32x4 acc[SN][SM] = {};
    for (int u = t.u0; u < t.u1; u += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (u + d >= t.u1) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if ((u + d) * 2 + s >= t.steps) break;
#pragma unroll
          for (int j = 0; j < SN; ++j)
#pragma unroll
            for (int i = 0; i < SM; ++i)
              acc[j][i] = mfma_scaled<0, 0>(__builtin_bit_cast(i32x4, x[d].b[s][j]),
                                            __builtin_bit_cast(i32x4, x[d].a[s][i]), acc[j][i], (int)x[d].sb[s][j],
                                            (int)x[d].sa[s][i]);
        }
        if (u + DEPTH + d < t.u1) load(t, u + DEPTH + d, x[d]);
      }
    }
    f32x4* part = s_part + par * waves * SN * SM * 64;
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int i = 0; i < SM; ++i) part[((wave * SN + j) * SM + i) * 64 + lane] = acc[j][i];
    // every wave's sums and the next tile; the sums of the tile before were
    // read before the barrier, so that two sets are enough
    __syncthreads();
    void* const C = t.C;
    const int M = t.M, N = t.N, m0 = t.m0, n0 = t.n0;
    v = __builtin_amdgcn_readfirstlane(s_tile[par ^ 1]);
    ++it;
    // Tiles of 16 columns have the next one's first units on their way
    // meanwhile (1 x 2048 x 8192 8.7 -> 7.7 us); at 32 columns the registers that
    // holds cost more than it hides (1 x 28672 x 8192 31.6 -> 33.1).
    if (SN == 1 && v >= 0) begin(v);
    for (int q = wave; q < SN * SM; q += waves) {
      f32x4 s = part[q * 64 + lane];
      for (int w = 1; w < waves; ++w) s += part[(w * SN * SM + q) * 64 + lane];
      const int64_t m = m0 + (q % SM) * 16 + l16, n = n0 + (q / SM) * 16 + 4 * kb;
      if (m >= M) continue;
      if (P.out_f32) {
        store_f32x4(static_cast<float*>(C) + m * N, n, N, s);
      } else {
        unsigned short* row = static_cast<unsigned short*>(C) + m * N;
        const unsigned lo = pack_bf16x2(s[0], s[1]), hi = pack_bf16x2(s[2], s[3]);
        if (n + 4 <= N) {
          *reinterpret_cast<u32x2_a2*>(row + n) = u32x2{lo, hi};
        } else {
          if (n < N) row[n] = (unsigned short)lo;
          if (n + 1 < N) row[n + 1] = (unsigned short)(lo >> 16);
          if (n + 2 < N) row[n + 2] = (unsigned short)hi;
        }
      }
    }
    if (SN != 1 && v >= 0) begin(v);
  }
  if (witness && tid == 0) {
    P.w.t_start[prog] = t_start;
    P.w.t_end[prog] = wall_ticks();
    P.w.cycles[prog] = shader_cycles() - c_start;
    P.w.hw_id[prog] = hw_placement();
    P.w.n_tiles[prog] = it;
  }
}

// --------------------------------------------------------------- instances

constexpr int kDevices = 64;

// A built tile: its kernels (one problem, several), threads and LDS.
struct Instance {
  int bm, bn;
  int threads, lds;
  void (*kern[2])(GemmParams);
  // resident workgroups per CU, by kernel and device; 0: not asked for yet (the
  // question and the LDS limit it sets cost microseconds of a short call)
  mutable std::atomic<int> resident[2][kDevices] = {};
};

template <int BM, int BN, int NST, int WN>
Instance tiled() {
  return {BM, BN, 128 * WN, Shape<BM, BN, NST, WN>::LDS_BYTES,
          {gemm_fp4_kernel<BM, BN, NST, WN, false>, gemm_fp4_kernel<BM, BN, NST, WN, true>}};
}
template <int SM, int SN, int DEPTH>
Instance skinny(int waves) {
  return {SM * 16, SN * 16, waves * 64, 2 * waves * SM * SN * 1024,
          {gemm_fp4_skinny_kernel<SM, SN, DEPTH, false>, gemm_fp4_skinny_kernel<SM, SN, DEPTH, true>}};
}

const Instance* instance(int bm, int bn, bool few) {
  static const Instance all[] = {
      tiled<256, 256, 2, 4>(), tiled<256, 128, 3, 2>(), tiled<128, 128, 2, 2>(),
      skinny<1, 1, 4>(8),      skinny<1, 2, 4>(4),      skinny<2, 2, 2>(4),       skinny<4, 2, 2>(4),
  };
  // At most one tile per CU: no second workgroup there covers the waits for
  // memory of a two-stage ring (512 x 8192 x 8192 33.1 -> 26.6 us, 128 x 28672 x
  // 8192 47.1 -> 36.8; with several tiles per CU two workgroups are faster, 8192^3
  // 340 against 360 us).
  static const Instance deep = tiled<128, 128, 3, 2>();
  if (few && bm == deep.bm && bn == deep.bn) return &deep;
  for (const Instance& i : all)
    if (i.bm == bm && i.bn == bn) return &i;
  return nullptr;
}

}  // namespace

bool gemm_fp4_tile_supported(int bm, int bn, int bk) { return bk == BK && instance(bm, bn, false) != nullptr; }

// Offsets of one tile's operand panels, and of two groups' scales, within 31
// bits (C is addressed with 64).
bool gemm_fp4_eligible(int bm, int bn, long long M, long long N, long long K) {
  const long long rows = bm > bn ? bm : bn;
  return rows * (K / 2) < (1LL << 31) && M < (1LL << 28) && N < (1LL << 28);
}

// The tile of the least estimated time: the rounds of tiles times what a CU
// needs for one, us for a 256-deep slab and for the stores (measured with all
// CUs busy: 256 x 256 2.0 and 5, 256 x 128 1.15 and 5, two workgroups of 128 x
// 128 1.3 and 4, one of them 0.75 and 4).  256 x 256 / 256 x 128 / 128 x 128
// measured: 8192^3 250 / 288 / 296 us, 4096^3 41 / 45 / 46, 2048 x 4096 x 4096
// 32 / 27 / 26, 1024 x 8192 x 8192 53 / 42 / 44, 512 x 8192 x 8192 47 / 34 / 27,
// 3000 x 7000 x 2048 to fp32 44 / 46 / 47, 700 x 5000 x 1408 19 / 18 / 12.
// Up to 64 rows the streaming kernel, unless more than half of the CUs get a
// 128 x 128 tile: past 16 rows its re-reading of A costs more than the tile's
// idle rows (64 x 28672 x 8192 65.8 against 35.4 us, 64 x 8192 x 8192 18.3
// against 23.9).  Tiles of 16 columns and eight waves while every tile has a CU
// (1 x 4096 x 14336 11.3 us against 14.2 with 32 columns and four; 1 x 8192 x 8192
// 14.1 against 10.8).
void gemm_fp4_default_tile(long long M, long long N, long long K, int cus, int& bm, int& bn, int& bk) {
  bk = BK;
  auto tiles = [&](int m, int n) { return (M + m - 1) / m * ((N + n - 1) / n); };
  if (M <= 16 || (M <= 64 && 2 * tiles(128, 128) <= cus)) {
    bm = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    bn = bm == 16 && N <= 16LL * cus ? 16 : 32;
    return;
  }
  auto rounds = [](long long t, long long slots) { return (double)((t + slots - 1) / slots); };
  const long long t = tiles(128, 128);
  const double slabs = (double)((K + BK - 1) / BK);
  const double big = rounds(tiles(256, 256), cus) * (2.0 * slabs + 5), mid = rounds(tiles(256, 128), cus) * (1.15 * slabs + 5);
  const double small = t <= cus ? 0.75 * slabs + 4 : rounds(t, 2LL * cus) * (1.3 * slabs + 4);
  bm = small < big && small < mid ? 128 : 256;
  bn = bm == 256 && big <= mid ? 256 : 128;
}

KernelInfo info_gemm_fp4(int bm, int bn, bool few, bool grouped) {
  const Instance* i = instance(bm, bn, few);
  if (!i) return KernelInfo{0, 0, 0};
  const int g = grouped ? 1 : 0;
  const void* kern = reinterpret_cast<const void*>(i->kern[g]);
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices)
    return KernelInfo{i->threads, i->lds, occupancy_of(kern, i->threads, i->lds)};
  int n = i->resident[g][dev].load(std::memory_order_acquire);
  if (n == 0) {
    n = occupancy_of(kern, i->threads, i->lds);
    i->resident[g][dev].store(n, std::memory_order_release);
  }
  return KernelInfo{i->threads, i->lds, n};
}

// After info_gemm_fp4 on the same device, which raises the kernel's LDS limit.
hipError_t launch_gemm_fp4(const GemmParams& p, int bm, int bn, bool few, hipStream_t stream) {
  const Instance* i = instance(bm, bn, few);
  if (!i) return hipErrorInvalidValue;
  hipLaunchKernelGGL(i->kern[p.ngemm > 0 ? 1 : 0], dim3(p.s.G), dim3(i->threads), i->lds, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
