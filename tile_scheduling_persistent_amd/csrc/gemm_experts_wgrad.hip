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
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kThreads = 256;
constexpr int BR = 64;  // rows per slab

// Physical 16-byte chunk of logical chunk c in row r: 32 lanes of a transposing
// read touch rows r .. r + 3 and r + 8 .. r + 11 at two adjacent chunks, 16
// chunks that this puts in distinct slots of a 256-byte window.
__device__ __forceinline__ int swz(int r, int c) { return c ^ (4 * (r & 3)) ^ (2 * ((r >> 3) & 1)); }

// Sixteen e4m3 codes times 2^(byte - 127), as bf16.
__device__ __forceinline__ void codes_bf16(u32x4 q, unsigned byte, u32x4& lo, u32x4& hi) {
  const float sc = scale_value(byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned w = i == 0 ? q[0] : i == 1 ? q[1] : i == 2 ? q[2] : q[3];
    const unsigned a = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, sc, false));
    const unsigned b = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, sc, true));
    if (i < 2) {
      lo[2 * i] = a;
      lo[2 * i + 1] = b;
    } else {
      hi[2 * (i - 2)] = a;
      hi[2 * (i - 2) + 1] = b;
    }
  }
}

// An operand's slab on its way: BR rows of W columns, 32 bytes of bf16 (two
// chunks) per thread and part.
template <int W, bool FP8>
struct Slab {
  static constexpr int PARTS = BR * W / 16 / kThreads;
  u32x4 q[PARTS][FP8 ? 1 : 2];
  unsigned byte[PARTS];
  // Rows r0 .. of `rows` (those past the end: zeros), columns c0 .. of the matrix
  // at `x` with `cols` columns (FP8: padded) and `ld` elements between rows.
  __device__ __forceinline__ void load(const void* x, const uint8_t* scale, int64_t ld, int64_t sld, int64_t row0, int r0,
                                       int rows, int c0, int cols) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = i * kThreads + threadIdx.x, r = at / (W / 16), c = c0 + at % (W / 16) * 16;
      const bool on = r0 + r < rows;
      const int64_t row = row0 + (on ? r0 + r : 0);
      if (FP8) {
        const bool in = on && c < cols;  // columns are whole groups
        q[i][0] = u32x4{0, 0, 0, 0};
        byte[i] = 0;
        if (in) {
          q[i][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(x) + row * ld + c);
          byte[i] = scale[(int64_t)(c >> 7) * sld + row];
        }
      } else {
        const unsigned short* p = static_cast<const unsigned short*>(x) + row * ld + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          q[i][h] = u32x4{0, 0, 0, 0};
          if (on && c + 8 * h + 8 <= cols) q[i][h] = *reinterpret_cast<const Quad<2>::type*>(p + 8 * h);
          else if (on && c + 8 * h < cols) {
            for (int e = 0; e < 7; ++e)
              if (c + 8 * h + e < cols) {
                const unsigned v = (unsigned)p[8 * h + e] << (16 * (e & 1));
                if (e < 2) q[i][h][0] |= v;
                else if (e < 4) q[i][h][1] |= v;
                else if (e < 6) q[i][h][2] |= v;
                else q[i][h][3] |= v;
              }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put(unsigned char* s) const {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = i * kThreads + threadIdx.x, r = at / (W / 16), c = at % (W / 16) * 2;
      u32x4 lo, hi;
      if (FP8) {
        codes_bf16(q[i][0], byte[i], lo, hi);
      } else {
        lo = q[i][0];
        hi = q[i][FP8 ? 0 : 1];
      }
      *reinterpret_cast<u32x4*>(s + r * W * 2 + swz(r, c) * 16) = lo;
      *reinterpret_cast<u32x4*>(s + r * W * 2 + swz(r, c + 1) * 16) = hi;
    }
  }
};

// A tile of BN x BK of one expert's gradient, four waves of BN/2 x BK/2.
template <int BN, int BK, bool DFP8>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(WgradParams p) {
  constexpr int TN = BN / 2, TK = BK / 2, SN = TN / 16, SK = TK / 16;
  constexpr int D_BYTES = BR * BN * 2, A_BYTES = BR * BK * 2;
  __shared__ __attribute__((aligned(1024))) unsigned char smem[D_BYTES + A_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wk = wave & 1;
  const int npn = (p.N + BN - 1) / BN, npk = (p.K + BK - 1) / BK;
  const int np = (p.N + 127) / 128 * 128, kp = (p.K + 127) / 128 * 128;
  const int64_t total = (int64_t)p.experts * npn * npk;

  // transposing reads: lane i of a group of 16 points at row i / 4 (+ 8 per
  // group), columns 4 (i % 4) .. of the block
  const int g = lane >> 4, i16 = lane & 15, a4 = i16 & 3, e4 = i16 >> 2;
  const int r_lane = g * 8 + e4;
  auto frag = [&](const unsigned char* s, int W, int col, int r0, i16x4 (&f)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + r_lane + 4 * h, n = col + 4 * a4;
      const unsigned char* at = s + r * W * 2 + swz(r, n >> 3) * 16 + 8 * (a4 & 1);
      f[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at);
    }
  };
  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int e = (int)(t / (npn * npk)), i = (int)(t - (int64_t)e * npn * npk);
    const int n0 = i / npk * BN, k0 = i % npk * BK;
    const ExpertRows rows = expert_rows(p.offsets, e, p.rows);
    f32x4 acc[SN][SK] = {};
    Slab<BN, DFP8> d;
    Slab<BK, true> a;
    auto load = [&](int r0) __attribute__((always_inline)) {
      d.load(p.D, p.sd, p.ldd, p.rows, rows.lo, r0, rows.n, n0, DFP8 ? np : p.N);
      a.load(p.A, p.sa, kp, p.rows, rows.lo, r0, rows.n, k0, kp);
    };
    if (rows.n > 0) load(0);
    for (int r0 = 0; r0 < rows.n; r0 += BR) {
      __syncthreads();
      d.put(smem);
      a.put(smem + D_BYTES);
      __syncthreads();
      if (r0 + BR < rows.n) load(r0 + BR);
#pragma unroll
      for (int s = 0; s < BR / 32; ++s) {
        i16x4 fd[SN][2], fa[SK][2];
#pragma unroll
        for (int j = 0; j < SN; ++j) frag(smem, BN, wn * TN + j * 16, s * 32, fd[j]);
#pragma unroll
        for (int j = 0; j < SK; ++j) frag(smem + D_BYTES, BK, wk * TK + j * 16, s * 32, fa[j]);
#pragma unroll
        for (int x = 0; x < SN; ++x)
#pragma unroll
          for (int y = 0; y < SK; ++y)
            acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, __builtin_shufflevector(fa[y][0], fa[y][1], 0, 1, 2, 3, 4, 5, 6, 7)),
                __builtin_bit_cast(bf16x8, __builtin_shufflevector(fd[x][0], fd[x][1], 0, 1, 2, 3, 4, 5, 6, 7)), acc[x][y], 0,
                0, 0);
      }
    }
    // lane: row n of the tile i16, columns k 4 g .. 4 g + 3 of each block
#pragma unroll
    for (int x = 0; x < SN; ++x) {
      const int n = n0 + wn * TN + x * 16 + i16;
      if (n >= p.N) continue;
      const int64_t at = ((int64_t)e * p.N + n) * p.K;
#pragma unroll
      for (int y = 0; y < SK; ++y)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = k0 + wk * TK + y * 16 + 4 * g + q;
          if (k >= p.K) continue;
          float v = acc[x][y][q];
          if (p.out_f32) {
            if (p.base) v += static_cast<const float*>(p.base)[at + k];
            static_cast<float*>(p.dB)[at + k] = v;
          } else {
            if (p.base)
              v += __builtin_bit_cast(float, (unsigned)static_cast<const unsigned short*>(p.base)[at + k] << 16);
            static_cast<unsigned short*>(p.dB)[at + k] = (unsigned short)pack_bf16x2(v, v);
          }
        }
    }
  }
}

}  // namespace

hipError_t launch_gemm_experts_wgrad(const WgradParams& p, int cus, hipStream_t stream) {
  if (p.sd)
    hipLaunchKernelGGL((wgrad_kernel<128, 128, true>), dim3(2 * cus), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((wgrad_kernel<128, 128, false>), dim3(2 * cus), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
