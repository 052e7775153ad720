// Persistent MXFP4 GEMM for gfx950: C[M][N] = A . B^T with A[M][K] and
// B[N][K] OCP e2m1 codes (two to a byte) and one e8m0 scale byte per 32
// consecutive k (SA[K/128][M][4], SB[K/128][N][4]), fp32 accumulate, C bf16
// or fp32.
//
// The scales enter v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies the 32
// k-values of row l % 16, block l / 16 of a 128-deep step as 16 bytes and the
// scale byte of exactly that block.
#include "common.hpp"
#include "gemm_device.hpp"

namespace pgk {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kFmtE2M1 = 4;  // f8f6f4 operand format code of e2m1

// One 64x64 tile per step of the schedule; four waves of 32x32, operands
// straight from memory.
template <bool WITNESS, bool GRP>
__global__ void __launch_bounds__(kThreads) gemm_fp4_kernel(GemmParams P) {
  __shared__ int s_tile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, kb = lane >> 4;
  const int prog = pgs::program_of(blockIdx.x, P.s.G, P.s.X, P.s.xcd_major);
  Walker walker(P.s, prog);
  if (WITNESS) walker.claim_row = P.w.claims + (size_t)prog * kMaxStealCounters;
  long long t_start = 0, c_start = 0;
  if (WITNESS && tid == 0) {
    t_start = wall_ticks();
    c_start = shader_cycles();
  }
  int it = 0, v = 0;
  for (;; ++it) {
    if (tid == 0) s_tile = it == 0 ? walker.first() : walker.next(v);
    __syncthreads();
    v = s_tile;
    __syncthreads();
    if (v < 0) break;
    if (tid == 0) {
      if (WITNESS) {
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
      for (int q = 1; q < P.ngemm; ++q)
        if (v >= P.gp[q].tile0) pr = P.gp[q];
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
    const int64_t m0 = (int64_t)pm * 64 + wm * 32, n0 = (int64_t)pn * 64 + wn * 32;
    const int64_t rowb = pr.K / 2;
    f32x4 acc[2][2] = {};
    for (int k = 0; k < pr.K; k += 128) {
      i32x8 a[2], b[2];
      int sa[2], sb[2];
      for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + i * 16 + l16, n = n0 + i * 16 + l16;
        i32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        sa[i] = sb[i] = 0;
        if (m < pr.M) {
          x = *reinterpret_cast<const i32x4*>(static_cast<const uint8_t*>(pr.A) + m * rowb + k / 2 + kb * 16);
          sa[i] = pr.sa[((int64_t)(k / 128) * pr.M + m) * 4 + kb];
        }
        if (n < pr.N) {
          y = *reinterpret_cast<const i32x4*>(static_cast<const uint8_t*>(pr.B) + n * rowb + k / 2 + kb * 16);
          sb[i] = pr.sb[((int64_t)(k / 128) * pr.N + n) * 4 + kb];
        }
        a[i] = i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
        b[i] = i32x8{y[0], y[1], y[2], y[3], 0, 0, 0, 0};
      }
      for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[i], acc[i][j], kFmtE2M1, kFmtE2M1,
                                                                       0, sb[j], 0, sa[i]);
    }
    // lane l holds row l % 16 of a block, columns 4*(l/16) .. +3
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j)
        for (int e = 0; e < 4; ++e) {
          const int64_t m = m0 + i * 16 + l16, n = n0 + j * 16 + 4 * kb + e;
          if (m >= pr.M || n >= pr.N) continue;
          if (P.out_f32)
            static_cast<float*>(pr.C)[m * pr.N + n] = acc[i][j][e];
          else
            static_cast<__bf16*>(pr.C)[m * pr.N + n] = (__bf16)acc[i][j][e];
        }
  }
  if (WITNESS && tid == 0) {
    P.w.t_start[prog] = t_start;
    P.w.t_end[prog] = wall_ticks();
    P.w.cycles[prog] = shader_cycles() - c_start;
    P.w.hw_id[prog] = hw_placement();
    P.w.n_tiles[prog] = it;
  }
}

}  // namespace

bool gemm_fp4_tile_supported(int bm, int bn, int bk) { return bm == 64 && bn == 64 && bk == 128; }

// Offsets of one tile's panels within 32 bits.
bool gemm_fp4_eligible(int bm, int bn, long long M, long long N, long long K) {
  const long long rows = bm > bn ? bm : bn;
  return rows * (K / 2) < (1LL << 31) && (long long)bm * N * 4 < (1LL << 31) && M < (1LL << 28) && N < (1LL << 28);
}

void gemm_fp4_default_tile(long long M, long long N, long long K, int cus, int& bm, int& bn, int& bk) {
  bm = 64;
  bn = 64;
  bk = 128;
}

KernelInfo info_gemm_fp4(int bm, int bn, bool grouped) {
  const void* k = grouped ? reinterpret_cast<const void*>(gemm_fp4_kernel<false, true>)
                          : reinterpret_cast<const void*>(gemm_fp4_kernel<false, false>);
  return KernelInfo{kThreads, 0, occupancy_of(k, kThreads, 0)};
}

hipError_t launch_gemm_fp4(const GemmParams& p, int bm, int bn, bool witness, hipStream_t stream) {
  const dim3 grid(p.s.G), threads(kThreads);
  if (p.ngemm > 0) {
    if (witness)
      hipLaunchKernelGGL((gemm_fp4_kernel<true, true>), grid, threads, 0, stream, p);
    else
      hipLaunchKernelGGL((gemm_fp4_kernel<false, true>), grid, threads, 0, stream, p);
  } else if (witness) {
    hipLaunchKernelGGL((gemm_fp4_kernel<true, false>), grid, threads, 0, stream, p);
  } else {
    hipLaunchKernelGGL((gemm_fp4_kernel<false, false>), grid, threads, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace pgk
