// e4m3 operands: rows with one scale per 128 columns, and weights with one scale
// per 128 x 128 block in both orientations.
#include "common.hpp"
#include "fp8_rows.hpp"

namespace pgk {
namespace {

// Rows: one pass, a block's largest magnitude among the 16 lanes that hold it.  Bound
// by memory: 5000 x 7000 fp32 35.1 us (5.0 TB/s; 38.1 with eight rows a wave).
template <int T, int RW>
__global__ void __launch_bounds__(kRowThreads) fp8_quant_kernel(Fp8QuantParams p) {
  constexpr int ROWS = 4 * RW;
  __shared__ TileScales<RW> s_scale;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t kp = (p.cols + 127) / 128 * 128, ctiles = (p.cols + kRowCols - 1) / kRowCols;
  const int64_t tiles = (p.rows + ROWS - 1) / ROWS * ctiles;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t row0 = rt * ROWS + wave * RW, c = ct * kRowCols + lane * 8;
    Vec8<T> v[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r < p.rows ? row0 + r : p.rows - 1;
      v[r] = vec8_load<T>(static_cast<const char*>(p.X) + row * p.ldx * size_of(T), c, p.cols);
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = vec8_get(v[r], e);
      unsigned byte;
      const u32x2_d o = e4m3_codes(x, byte);
      if (row0 + r < p.rows && c < kp) *reinterpret_cast<u32x2_d*>(p.Q + (row0 + r) * kp + c) = o;
      s_scale.put(lane, wave * RW + r, byte);
    }
    __syncthreads();
    s_scale.store(p.scale, ct * 4, kp / 128, rt * ROWS, p.rows, p.rows);
    __syncthreads();
  }
}

// Weights: a workgroup takes one block of 128 x 128.  Lane i % 16 of a row of
// lanes holds columns 8 i .. 8 i + 7 of eight consecutive rows: an 8 x 8 block of
// codes, which is transposed in registers and goes through LDS into rows of the
// transposed output.  Bound by memory: 16 x 4096 x 4096 bf16, both orientations, 1.07 GB
// in 200 us (5.4 TB/s).
// Byte of 8-byte piece `piece` of transposed row `row` in LDS: 16 lanes write one piece of
// every eighth row, and read one row's (rows 136 bytes apart, without the flip: 16 x 4096
// x 4096 fp32 298 us, so 294; 4 x 1408 x 2048 bf16 10.8, so 10.4).
__device__ __forceinline__ int piece_at(int row, int piece) { return row * 128 + (piece ^ (row >> 3)) * 8; }
template <int T>
__global__ void __launch_bounds__(256) fp8_quant_weights_kernel(Fp8WeightsParams p) {
  __shared__ __attribute__((aligned(16))) unsigned char s_t[128 * 128];
  __shared__ unsigned s_max[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t rp = (p.rows + 127) / 128, cp = (p.cols + 127) / 128, blocks = rp * cp;
  const int64_t total = p.experts * blocks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int64_t e = b / blocks, i = b - e * blocks, br = i / cp, bc = i - br * cp;
    const int r0 = (tid >> 4) * 8, c0 = (tid & 15) * 8;
    const char* x = static_cast<const char*>(p.X) + e * p.rows * p.cols * size_of(T);
    Vec8<T> v[8];
    unsigned amax = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t row = br * 128 + r0 + r;
      // rows past the end are empty: a row of no columns
      v[r] = vec8_load<T>(x + (row < p.rows ? row : 0) * p.cols * size_of(T), bc * 128 + c0, row < p.rows ? p.cols : 0);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) amax = max_u32(amax, vec8_amax(v[r]));
    amax = row16_max(amax);
#pragma unroll
    for (int d = 16; d < 64; d *= 2) amax = max_u32(amax, (unsigned)__shfl_xor((int)amax, d));
    if (lane == 0) s_max[wave] = amax;
    __syncthreads();
    amax = max_u32(max_u32(s_max[0], s_max[1]), max_u32(s_max[2], s_max[3]));
    const unsigned byte = scale_byte<E4M3>(amax, kRuleCeil);
    const float sc = scale_value(byte);
    u32x2_d q[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s16x2_d t = {0, 0};
        t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, vec8_get(v[r], 4 * h), vec8_get(v[r], 4 * h + 1), sc, false);
        t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, vec8_get(v[r], 4 * h + 2), vec8_get(v[r], 4 * h + 3), sc, true);
        q[r][h] = byte == 255u ? 0u : __builtin_bit_cast(unsigned, t);
      }
      const int64_t row = br * 128 + r0 + r;
      if (row < p.rows) *reinterpret_cast<u32x2_d*>(p.Q + ((e * p.rows + row) * cp + bc) * 128 + c0) = q[r];
    }
    if (tid == 0) p.scale[(e * rp + br) * cp + bc] = (uint8_t)byte;
    if (p.Qt) {
      // 4 x 4 bytes at a time: rows 4 a .., columns 4 h ..
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned t[4][2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const unsigned w0 = q[4 * a][h], w1 = q[4 * a + 1][h], w2 = q[4 * a + 2][h], w3 = q[4 * a + 3][h];
          const unsigned lo01 = __builtin_amdgcn_perm(w1, w0, 0x05010400u), hi01 = __builtin_amdgcn_perm(w1, w0, 0x07030602u);
          const unsigned lo23 = __builtin_amdgcn_perm(w3, w2, 0x05010400u), hi23 = __builtin_amdgcn_perm(w3, w2, 0x07030602u);
          t[0][a] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
          t[1][a] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
          t[2][a] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
          t[3][a] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<u32x2_d*>(s_t + piece_at(c0 + 4 * h + k, r0 >> 3)) = u32x2_d{t[k][0], t[k][1]};
      }
      if (tid == 0) p.scale_t[(e * cp + bc) * rp + br] = (uint8_t)byte;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = j * 16 + (tid >> 4), at = (tid & 15) * 8;
        const int64_t k = bc * 128 + row;
        if (k < p.cols)
          *reinterpret_cast<u32x2_d*>(p.Qt + ((e * p.cols + k) * rp + br) * 128 + at) =
              *reinterpret_cast<const u32x2_d*>(s_t + piece_at(row, at >> 3));
      }
    }
    __syncthreads();
  }
}

template <int T>
void quant_typed(const Fp8QuantParams& p, hipStream_t stream) {
  // four rows a wave where the tiles still fill the CUs twice over
  if (row_tiles(p.rows, p.cols, 4) >= 2 * p.cus)
    hipLaunchKernelGGL((fp8_quant_kernel<T, 4>), row_grid(row_tiles(p.rows, p.cols, 4)), dim3(kRowThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((fp8_quant_kernel<T, 1>), row_grid(row_tiles(p.rows, p.cols, 1)), dim3(kRowThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_fp8_quant(const Fp8QuantParams& p, hipStream_t stream) {
  if (p.type == kTypeF32)
    quant_typed<kTypeF32>(p, stream);
  else if (p.type == kTypeBF16)
    quant_typed<kTypeBF16>(p, stream);
  else
    quant_typed<kTypeF16>(p, stream);
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weights(const Fp8WeightsParams& p, hipStream_t stream) {
  const dim3 grid = row_grid(p.experts * ((p.rows + 127) / 128) * ((p.cols + 127) / 128));
  if (p.type == kTypeF32)
    hipLaunchKernelGGL(fp8_quant_weights_kernel<kTypeF32>, grid, dim3(256), 0, stream, p);
  else if (p.type == kTypeBF16)
    hipLaunchKernelGGL(fp8_quant_weights_kernel<kTypeBF16>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(fp8_quant_weights_kernel<kTypeF16>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
