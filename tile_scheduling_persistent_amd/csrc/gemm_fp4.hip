// Persistent MXFP4 GEMM for gfx950: C[M][N] = A . B^T with A[M][K] and
// B[N][K] OCP e2m1 codes (two to a byte) and one e8m0 scale byte per 32
// consecutive k (SA[K/128][M][4], SB[K/128][N][4]), fp32 accumulate, C bf16
// or fp32.
//
// The scales enter v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies the 32
// k-values of row l % 16, block l / 16 of a 128-deep step as 16 bytes and the
// scale byte of exactly that block.  C comes out transposed in the lanes (the
// B rows are the first operand): lane l holds row l % 16 of a 16x16 block of
// C, columns 4 * (l / 16) .. +3.
//
// Two kernels:
//  * gemm_fp4_kernel, tiles staged through LDS: bound by the matrix cores and,
//    on data that is not all zeros, by the power they draw.
//  * gemm_fp4_skinny_kernel for up to 64 rows: bound by the bytes of B, which
//    each wave streams straight into registers; the waves of a workgroup split
//    K and add their sums in LDS.
#include <type_traits>
#include <utility>

#include "common.hpp"
#include "gemm_device.hpp"

namespace pgk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
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

// Columns c .. c + 3 (fp32) or c .. c + 7 (bf16) of a row of C that ends at n.
// Rows of C start on any element; stores of any alignment are single
// instructions.
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
__device__ __forceinline__ void store_f32x4(float* row, int64_t c, int64_t n, f32x4 v) {
  if (c + 4 <= n) {
    *reinterpret_cast<u32x4_a4*>(row + c) = __builtin_bit_cast(u32x4, v);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (c + e < n) row[c + e] = v[e];
  }
}
__device__ __forceinline__ void store_bf16x8(unsigned short* row, int64_t c, int64_t n, u32x4 v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u32x4_a2*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (c + e < n) row[c + e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
  }
}

// ------------------------------------------------------------ tiles in LDS
//
// Four waves, 2 x 2, each TM x TN of the tile.  A slab is 256 deep: 128 bytes
// of each row of A and of B, so every global access is whole 128-byte lines,
// and the scale words of its two 128-deep groups.  A ring of NST slabs in LDS
// is filled by hand-issued buffer_load ... lds (gemm_device.hpp); the loads of
// slab g + NST - 1 are spread over the first MFMAs of a slab period, across
// tiles too.
//
// Both operands have 128-byte rows in LDS, chunk-swizzled like A of the fp8
// kernel: a ds_read_b128 is served 16 lanes at a time, here 16 consecutive
// rows at one 16-byte chunk, which the XOR with (row >> 1) spreads over the 16
// slots of a 256-byte window.
//
// Scales: the load of the scale words permutes rows so that the words of row
// l of all the wave's 16-row blocks stand side by side in LDS: a lane reads
// four blocks' words with one ds_read_b128 and gathers its own byte of each
// into one register (v_perm), from which the MFMA selects by opsel.  Byte
// reads per block would be four times the LDS instructions.
template <int BM, int BN, int NST_>
struct Shape {
  static constexpr int NST = NST_;
  static constexpr int TM = BM / 2, TN = BN / 2;
  static constexpr int SM = TM / 16, SN = TN / 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SA_BYTES = BM * 8, SB_BYTES = BN * 8;  // two groups of words
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int LDS_BYTES = NST * STAGE + 16;  // + first tile, next tile [2]
  static constexpr int NA = BM / 32, NB = BN / 32;    // 1 KB operand loads per wave per slab
  static constexpr int NSA = BM / 128, NSB = BN / 128;  // 256-byte scale loads per wave per slab
  static constexpr int NL = NA + NB + NSA + NSB;
  static constexpr int NMF = SM * SN;                 // MFMAs per 128-deep step
  static constexpr int NRD = SM + SN + SM / 4 + SN / 4;
  static_assert(SM % 4 == 0 && SN % 4 == 0, "scale bytes gathered four blocks at a time");
  static_assert(BM % 128 == 0 && BN % 128 == 0 && NA % 2 == 0 && NB % 2 == 0, "whole loads per wave");
};

template <int BM, int BN, int NST, bool GRP>
__global__ void __launch_bounds__(kThreads) gemm_fp4_kernel(GemmParams P) {
  using S = Shape<BM, BN, NST>;
  constexpr int NA = S::NA, NB = S::NB, NO = NA + NB, NL = S::NL, NMF = S::NMF, NRD = S::NRD;
  constexpr int SM = S::SM, SN = S::SN;
  // Of a period's 2 * NMF MFMA positions, the loads take the first SPREAD, and
  // the next step's LDS reads the first RSPREAD of each step's.
  constexpr int SPREAD = NL > NMF ? 2 * NMF : NMF;
  constexpr int RSPREAD = NRD > NMF * 3 / 4 ? NMF : NMF * 3 / 4;

  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  int* s_first = reinterpret_cast<int*>(smem + NST * S::STAGE);
  int* s_next = s_first + 1;  // [2]: the loader's next tile, by claim parity

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, kb = lane >> 4;
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
  // row 8q + p / 8, LDS chunk p % 8, global chunk (p % 8) ^ ((row >> 1) & 7).
  // Instruction i of wave w is q = w * NA + i (NA even), so the chunk depends
  // on the lane and on i's parity only.
  const int r8 = lane >> 3;
  const unsigned chunk0 = (unsigned)((lane & 7) ^ ((r8 >> 1) & 7));  // q even; odd q: ^ 4
  unsigned aoff = 0, boff = 0;  // instruction 0, chunk excluded
  unsigned astep = 0;           // 8 rows
  auto lane_offsets = [&](int Kx) {
    const unsigned rowb = (unsigned)Kx >> 1;
    aoff = (unsigned)(wave * NA * 8 + r8) * rowb;
    boff = (unsigned)(wave * NB * 8 + r8) * rowb;
    astep = 8u * rowb;
  };
  lane_offsets(Kl);
  // Scales: LDS dword d of the A region (group, half of the tile, l16, block)
  // holds the word of row half * TM + block * 16 + l16; likewise B.
  auto scale_row = [&](int d, int B, int T, int SB, int& grp, int& row) {
    grp = d / B;
    const int rem = d % B, half = rem / T, e = rem % T;
    row = half * T + (e % SB) * 16 + e / SB;
  };
  const unsigned lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));

  // LDS reads: step s, block i: row (block origin) + l16, chunk 4 s + kb.
  unsigned rd_a[2], rd_b[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const unsigned c = (unsigned)((4 * s + kb) ^ ((l16 >> 1) & 7));
    rd_a[s] = (unsigned)((wm * S::TM + l16) * 128) + c * 16u;
    rd_b[s] = (unsigned)(S::A_BYTES + (wn * S::TN + l16) * 128) + c * 16u;
  }
  const unsigned rd_sa = (unsigned)(S::A_BYTES + S::B_BYTES + (wm * S::TM + l16 * SM) * 4);
  const unsigned rd_sb = (unsigned)(S::A_BYTES + S::B_BYTES + S::SA_BYTES + (wn * S::TN + l16 * SN) * 4);
  // v_perm selectors: byte kb of two words into the low or the high half
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
  rsrc_words_t rA, rB, rSA, rSB;
  unsigned long long a_ptr = 0, b_ptr = 0;
  unsigned a_rec = 0, b_rec = 0;
  unsigned half0 = 0, half1 = 0;  // kOob in lanes whose chunk is past K (even, odd instructions)
  unsigned soa[S::NSA], sob[S::NSB];

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
    int grp, row;
#pragma unroll
    for (int i = 0; i < S::NSA; ++i) {
      scale_row((wave * S::NSA + i) * 64 + lane, BM, S::TM, SM, grp, row);
      soa[i] = lm0 + row < Ml ? (unsigned)(grp * Ml + row) * 4u : kOob;
    }
#pragma unroll
    for (int i = 0; i < S::NSB; ++i) {
      scale_row((wave * S::NSB + i) * 64 + lane, BN, S::TN, SN, grp, row);
      sob[i] = ln0 + row < Nl ? (unsigned)(grp * Nl + row) * 4u : kOob;
    }
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
    // the second half of an odd last slab is past K: its chunks are past
    // every range, its scale words (the other group's rows) likewise
    const bool odd = k0 + 128 >= Kl;
    const unsigned hi0 = (chunk0 & 4u) ? kOob : 0u;
    half0 = odd ? hi0 : 0u;
    half1 = odd ? hi0 ^ kOob : 0u;
    const int grp = k0 >> 7, ng = odd ? 1 : 2;
    rSA = rsrc_words_u64(reinterpret_cast<unsigned long long>(SAl + ((size_t)grp * Ml + lm0) * 4),
                         load ? (unsigned)(ng * Ml - lm0) * 4u : 0u);
    rSB = rsrc_words_u64(reinterpret_cast<unsigned long long>(SBl + ((size_t)grp * Nl + ln0) * 4),
                         load ? (unsigned)(ng * Nl - ln0) * 4u : 0u);
  };

  auto dma = [&](int st, int d) PGK_INLINE {
    const unsigned sb = lds0 + (unsigned)(st * S::STAGE);
    if (d < NA) {
      const unsigned ch = (d & 1) ? (chunk0 ^ 4u) : chunk0;
      load_lds16(rA, sb + (unsigned)((wave * NA + d) * 1024),
                 (aoff + (unsigned)d * astep + ch * 16u) | ((d & 1) ? half1 : half0));
    } else if (d < NO) {
      const int e = d - NA;
      const unsigned ch = (e & 1) ? (chunk0 ^ 4u) : chunk0;
      load_lds16(rB, sb + (unsigned)(S::A_BYTES + (wave * NB + e) * 1024),
                 (boff + (unsigned)e * astep + ch * 16u) | ((e & 1) ? half1 : half0));
    } else if (d < NO + S::NSA) {
      load_lds4(rSA, sb + (unsigned)(S::A_BYTES + S::B_BYTES + (wave * S::NSA + d - NO) * 256), soa[d - NO]);
    } else {
      const int e = d - NO - S::NSA;
      load_lds4(rSB, sb + (unsigned)(S::A_BYTES + S::B_BYTES + S::SA_BYTES + (wave * S::NSB + e) * 256), sob[e]);
    }
  };

  f32x4 acc[SN][SM];
  i32x4 aq[2][SM], bq[2][SN];               // fragments, by step
  u32x4 wa[2][SM / 4], wb[2][SN / 4];       // scale words, by step
  int sa[SM / 4], sb[SN / 4];               // gathered scale bytes of the step on the matrix cores

  // LDS read r of step s: scale words, then B block 0, the A blocks, the other
  // B blocks (the order the MFMAs consume them).
  auto read = [&](int st, int s, int r) PGK_INLINE {
    const unsigned char* p = smem + st * S::STAGE;
    constexpr int NW = SM / 4 + SN / 4;
    if (r < SM / 4) {
      wa[s][r] = *reinterpret_cast<const u32x4*>(p + rd_sa + s * BM * 4 + r * 16);
    } else if (r < NW) {
      wb[s][r - SM / 4] = *reinterpret_cast<const u32x4*>(p + rd_sb + s * BN * 4 + (r - SM / 4) * 16);
    } else if (r == NW) {
      bq[s][0] = *reinterpret_cast<const i32x4*>(p + rd_b[s]);
    } else if (r <= NW + SM) {
      aq[s][r - NW - 1] = *reinterpret_cast<const i32x4*>(p + rd_a[s] + (r - NW - 1) * 2048);
    } else {
      bq[s][r - NW - SM] = *reinterpret_cast<const i32x4*>(p + rd_b[s] + (r - NW - SM) * 2048);
    }
  };
  auto gather = [&](u32x4 w) {
    return (int)(__builtin_amdgcn_perm(w[1], w[0], sel_lo) | __builtin_amdgcn_perm(w[3], w[2], sel_hi));
  };
  auto scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < SM / 4; ++i) sa[i] = gather(wa[s][i]);
#pragma unroll
    for (int i = 0; i < SN / 4; ++i) sb[i] = gather(wb[s][i]);
  };
  auto mfma = [&](auto sc, auto jc) PGK_INLINE {
    constexpr int s = sc, sn = jc / SM, sm = jc % SM;
    acc[sn][sm] = mfma_scaled<sn % 4, sm % 4>(bq[s][sn], aq[s][sm], acc[sn][sm], sb[sn / 4], sa[sm / 4]);
  };
  // Step s on the matrix cores; the other step's reads (of stage st_rd) and
  // the loads that fall on this half of the period.
  auto step = [&](auto sc, int st_rd, int st_dma) PGK_INLINE {
    static_for<NMF>([&](auto jc) PGK_INLINE {
      constexpr int s = sc, j = jc;
      mfma(sc, jc);
      static_for<NRD>([&](auto rc) PGK_INLINE {
        if constexpr (rc * RSPREAD / NRD == j) read(st_rd, s ^ 1, rc);
      });
      static_for<NL>([&](auto dc) PGK_INLINE {
        if constexpr (dc * SPREAD / NL == (s == 1 ? j : NMF + j)) dma(st_dma, dc);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  auto epilogue = [&](int m0, int n0) {
    const int64_t N = Nc;
    const int mb = m0 + wm * S::TM + l16, nb = n0 + wn * S::TN;
#pragma unroll
    for (int i = 0; i < SM; ++i) {
      const int m = mb + i * 16;
      if (m >= Mc) continue;
      if (P.out_f32) {
        float* row = static_cast<float*>(Cc) + (int64_t)m * N;
#pragma unroll
        for (int j = 0; j < SN; ++j) store_f32x4(row, nb + j * 16 + 4 * kb, N, acc[j][i]);
      } else {
        unsigned short* row = static_cast<unsigned short*>(Cc) + (int64_t)m * N;
        // Two neighbouring blocks at a time: v_permlane16_swap trades the odd
        // 16-lane rows of one for the even rows of the other, which leaves each
        // lane eight consecutive columns.
#pragma unroll
        for (int j = 0; j < SN; j += 2) {
          const f32x4 a = acc[j][i], b = acc[j + 1][i];
          const auto s0 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), false, false);
          const auto s1 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[2], a[3]), pack_bf16x2(b[2], b[3]), false, false);
          store_bf16x8(row, nb + (j + (kb & 1)) * 16 + 4 * (kb & 2), N, u32x4{s0[0], s1[0], s0[1], s1[1]});
        }
      }
    }
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
      for (int i = 0; i < SM; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // A period per slab: the barrier, step 1 of the slab before (fragments in
    // registers) while step 0 of this one is read, then step 0 while step 1 is
    // read.  The tile's first slab has no step before it.
    {
      slab_start();
      const int st = g % NST, st_dma = st == 0 ? NST - 1 : st - 1;
#pragma unroll
      for (int r = 0; r < NRD; ++r) read(st, 0, r);
      __builtin_amdgcn_sched_barrier(0);
      prep();
#pragma unroll
      for (int d = 0; d < NL; ++d)
        if (d * SPREAD / NL < NMF) dma(st_dma, d);
      scales(0);
      __builtin_amdgcn_sched_barrier(0);
      step(step0, st, st_dma);
      scales(1);
      ++g;
    }
    for (int ck = 1; ck < cnk; ++ck) {
      slab_start();
      const int st = g % NST, st_dma = st == 0 ? NST - 1 : st - 1;
      prep();
      __builtin_amdgcn_sched_barrier(0);
      step(step1, st, st_dma);
      scales(0);
      __builtin_amdgcn_sched_barrier(0);
      step(step0, st, st_dma);
      scales(1);
      __builtin_amdgcn_sched_barrier(0);
      ++g;
    }
    static_for<NMF>([&](auto jc) PGK_INLINE { mfma(step1, jc); });
    // all of them before the epilogue's branches, whose blocks they would
    // otherwise move into, each wait then for one block's results
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int i = 0; i < SM; ++i) asm volatile("" : "+a"(acc[j][i]));
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
  f32x4* s_part = reinterpret_cast<f32x4*>(smem);  // [waves][SN][SM][64]
  __shared__ int s_tile;
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
  struct Unit {
    u32x4 b[2][SN], a[2][SM];
    unsigned sb[2][SN], sa[2][SM];
  };
  int it = 0, v = 0;
  for (;; ++it) {
    if (tid == 0) s_tile = it == 0 ? walker.first() : walker.next(v);
    __syncthreads();
    v = __builtin_amdgcn_readfirstlane(s_tile);
    if (v < 0) break;
    if (tid == 0) {
      if (witness) {
        atomicAdd(P.w.visits + v, 1);
        P.w.owner[v] = prog;
        P.w.order[v] = it;
      }
      if (is_straggler(P.s, prog)) spin_ns(P.s.straggler_ns, P.s.wall_khz);
    }
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
    const int m0 = pm * 16 * SM, n0 = pn * 16 * SN;
    const int rowb = pr.K >> 1, steps = pr.K >> 7;
    const int ra = pr.M - m0 < 16 * SM ? pr.M - m0 : 16 * SM, rb = pr.N - n0 < 16 * SN ? pr.N - n0 : 16 * SN;
    // rows past the operands read as zeros (range checks)
    const auto rA = rsrc(static_cast<const uint8_t*>(pr.A) + (size_t)m0 * rowb, (unsigned)(ra * rowb));
    const auto rB = rsrc(static_cast<const uint8_t*>(pr.B) + (size_t)n0 * rowb, (unsigned)(rb * rowb));
    const unsigned off = (unsigned)l16 * (unsigned)rowb + (unsigned)kb * 16u;
    const unsigned soff = (unsigned)(l16 * 4 + kb);
    auto load = [&](int u, Unit& x) PGK_INLINE {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int st = u * 2 + s;
        const bool in = st < steps;  // uniform
        const unsigned at = in ? off + (unsigned)st * 64u : kOob;
        const auto rSA = rsrc(pr.sa + ((size_t)(in ? st : 0) * pr.M + m0) * 4, (unsigned)(ra * 4));
        const auto rSB = rsrc(pr.sb + ((size_t)(in ? st : 0) * pr.N + n0) * 4, (unsigned)(rb * 4));
#pragma unroll
        for (int j = 0; j < SN; ++j) {
          x.b[s][j] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rB, at + (unsigned)(j * 16) * (unsigned)rowb, 0, 0));
          x.sb[s][j] = __builtin_amdgcn_raw_buffer_load_b8(rSB, soff + j * 64, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < SM; ++i) {
          x.a[s][i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rA, at + (unsigned)(i * 16) * (unsigned)rowb, 0, 0));
          x.sa[s][i] = __builtin_amdgcn_raw_buffer_load_b8(rSA, soff + i * 64, 0, 0);
        }
      }
    };
    f32x4 acc[SN][SM] = {};
    // the wave's units: a consecutive stretch, so that a row's lines are read
    // one after the other
    const int units = (steps + 1) >> 1, u0 = units * wave / waves, u1 = units * (wave + 1) / waves;
    Unit x[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (u0 + d < u1) load(u0 + d, x[d]);
    for (int u = u0; u < u1; u += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (u + d >= u1) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if ((u + d) * 2 + s >= steps) break;
#pragma unroll
          for (int j = 0; j < SN; ++j)
#pragma unroll
            for (int i = 0; i < SM; ++i)
              acc[j][i] = mfma_scaled<0, 0>(__builtin_bit_cast(i32x4, x[d].b[s][j]),
                                            __builtin_bit_cast(i32x4, x[d].a[s][i]), acc[j][i], (int)x[d].sb[s][j],
                                            (int)x[d].sa[s][i]);
        }
        if (u + DEPTH + d < u1) load(u + DEPTH + d, x[d]);
      }
    }
#pragma unroll
    for (int j = 0; j < SN; ++j)
#pragma unroll
      for (int i = 0; i < SM; ++i) s_part[((wave * SN + j) * SM + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    for (int q = wave; q < SN * SM; q += waves) {
      f32x4 s = s_part[q * 64 + lane];
      for (int w = 1; w < waves; ++w) s += s_part[(w * SN * SM + q) * 64 + lane];
      const int64_t m = m0 + (q % SM) * 16 + l16, n = n0 + (q / SM) * 16 + 4 * kb;
      if (m >= pr.M) continue;
      if (P.out_f32) {
        store_f32x4(static_cast<float*>(pr.C) + m * pr.N, n, pr.N, s);
      } else {
        unsigned short* row = static_cast<unsigned short*>(pr.C) + m * pr.N;
        const unsigned lo = pack_bf16x2(s[0], s[1]), hi = pack_bf16x2(s[2], s[3]);
        typedef unsigned u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
        if (n + 4 <= pr.N) {
          *reinterpret_cast<u32x2_a2*>(row + n) = u32x2_a2{lo, hi};
        } else {
          if (n < pr.N) row[n] = (unsigned short)lo;
          if (n + 1 < pr.N) row[n + 1] = (unsigned short)(lo >> 16);
          if (n + 2 < pr.N) row[n + 2] = (unsigned short)hi;
        }
      }
    }
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

// A built tile: its kernels (one problem, several), threads and LDS.
struct Instance {
  int bm, bn;
  int threads, lds;
  void (*kern[2])(GemmParams);
};

template <int BM, int BN, int NST>
Instance tiled() {
  return {BM, BN, kThreads, Shape<BM, BN, NST>::LDS_BYTES,
          {gemm_fp4_kernel<BM, BN, NST, false>, gemm_fp4_kernel<BM, BN, NST, true>}};
}
template <int SM, int SN, int DEPTH>
Instance skinny(int waves) {
  return {SM * 16, SN * 16, waves * 64, waves * SM * SN * 1024,
          {gemm_fp4_skinny_kernel<SM, SN, DEPTH, false>, gemm_fp4_skinny_kernel<SM, SN, DEPTH, true>}};
}

const Instance* instance(int bm, int bn) {
  static const Instance all[] = {
      tiled<256, 256, 2>(), tiled<256, 128, 3>(), tiled<128, 128, 2>(),
      skinny<1, 1, 4>(8),   skinny<1, 2, 4>(4),   skinny<2, 2, 2>(4),   skinny<4, 2, 2>(4),
  };
  for (const Instance& i : all)
    if (i.bm == bm && i.bn == bn) return &i;
  return nullptr;
}

}  // namespace

bool gemm_fp4_tile_supported(int bm, int bn, int bk) { return bk == BK && instance(bm, bn) != nullptr; }

// Offsets of one tile's operand panels, and of two groups' scales, within 31
// bits (C is addressed with 64).
bool gemm_fp4_eligible(int bm, int bn, long long M, long long N, long long K) {
  const long long rows = bm > bn ? bm : bn;
  return rows * (K / 2) < (1LL << 31) && M < (1LL << 28) && N < (1LL << 28);
}

void gemm_fp4_default_tile(long long M, long long N, long long K, int cus, int& bm, int& bn, int& bk) {
  bk = BK;
  if (M <= 64) {
    bm = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    bn = bm == 16 && N <= 16LL * 4 * cus ? 16 : 32;
    return;
  }
  bm = M <= 128 ? 128 : 256;
  bn = bm == 128 ? 128 : (M + 255) / 256 * ((N + 255) / 256) >= cus ? 256 : 128;
  if (bm == 256 && bn == 128 && (M + 255) / 256 * ((N + 127) / 128) < cus) bm = 128;
}

KernelInfo info_gemm_fp4(int bm, int bn, bool grouped) {
  const Instance* i = instance(bm, bn);
  if (!i) return KernelInfo{0, 0, 0};
  return KernelInfo{i->threads, i->lds,
                    occupancy_of(reinterpret_cast<const void*>(i->kern[grouped ? 1 : 0]), i->threads, i->lds)};
}

hipError_t launch_gemm_fp4(const GemmParams& p, int bm, int bn, hipStream_t stream) {
  const Instance* i = instance(bm, bn);
  if (!i) return hipErrorInvalidValue;
  auto kern = i->kern[p.ngemm > 0 ? 1 : 0];
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, i->lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(p.s.G), dim3(i->threads), i->lds, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
