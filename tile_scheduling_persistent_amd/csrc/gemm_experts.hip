// C[r][n] = sum over k of A[r][k] B_e[n][k], e the expert of row r: A e4m3 with
// one e8m0 scale per 128 k of a row, B e4m3 with one per block of 128 n x 128 k,
// fp32 accumulate, C bf16 or fp32.
//
// To bf16 the products run on the scaled e4m3 MFMA.  It keeps a product to 2^-13
// of the largest of eight that it adds first (measured: 2^2 beside 2^16 is lost
// there, 2^3 is not), which bf16's 2^-8 hides but fp32 does not: a result's error
// was 1.5e-5 of its size at any K.  To fp32 the elements are therefore multiplied
// by their scales, exactly, into bf16 and go through the bf16 MFMA, which adds
// their exact products in fp32 at half the rate.
//
// The rows are sorted by expert and the experts' row counts are in device memory:
// each program of the grid adds up the tiles that the experts have and walks the
// tiles with a stride of the grid.
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
typedef float f32x4 __attribute__((ext_vector_type(4)));
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

}  // namespace

hipError_t launch_gemm_experts(const ExpertsParams& p, int cus, hipStream_t stream) {
  const int lds = (3 * p.experts + 1) * (int)sizeof(int);
  if (p.out_f32)
    hipLaunchKernelGGL((gemm_experts_stream_kernel<1, 1, 4, 8, true>), dim3(2 * cus), dim3(512), lds, stream, p);
  else
    hipLaunchKernelGGL((gemm_experts_stream_kernel<1, 1, 4, 8, false>), dim3(2 * cus), dim3(512), lds, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
