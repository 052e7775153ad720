// MXFP4 operands: quantisation of a matrix along its rows or (transposed) its
// columns, and the way back.
#include "common.hpp"
#include "mx_device.hpp"

namespace pgk {
namespace {

// One thread per block of 32.
template <int T>
__global__ void __launch_bounds__(256) quant_kernel(QuantParams p) {
  const int64_t len = p.transpose ? p.rows : p.cols, lines = p.transpose ? p.cols : p.rows;
  const int64_t groups = (len + 127) / 128;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t blk = t % (groups * 4), line = t / (groups * 4);
  if (line >= lines) return;
  const int64_t step = p.transpose ? p.ldx : 1, base = p.transpose ? line : line * p.ldx;
  float x[32];
  unsigned amax = 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int64_t k = blk * 32 + e;
    x[e] = k < len ? load_elem<T>(p.X, base + k * step) : 0.0f;
    const unsigned b = __builtin_bit_cast(unsigned, x[e]) & 0x7fffffffu;
    amax = b > amax ? b : amax;
  }
  const unsigned byte = scale_byte<E2M1>(amax, p.rule);
  const float s = scale_value(byte);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    Vec8<kTypeF32> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.q[e >> 2][e & 3] = __builtin_bit_cast(unsigned, x[8 * q + e]);
    reinterpret_cast<unsigned*>(p.Q + line * groups * 64 + blk * 16)[q] = byte == 255u ? 0u : vec8_e2m1(v, s);
  }
  p.scale[((blk >> 2) * lines + line) * 4 + (blk & 3)] = (uint8_t)byte;
}

// One thread per eight values.
template <int T>
__global__ void __launch_bounds__(256) dequant_kernel(DequantParams p) {
  const int64_t groups = (p.cols + 127) / 128;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = (p.cols + 7) / 8, row = t / per, c = (t % per) * 8;
  if (row >= p.rows) return;
  const unsigned codes = *reinterpret_cast<const unsigned*>(p.Q + row * groups * 64 + c / 2);
  float x[8];
  e2m1_values(codes, p.scale[((c >> 7) * p.rows + row) * 4 + ((c >> 5) & 3)], x);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < p.cols) store_elem<T>(p.Y, row * p.ldy + c + e, x[e]);
}

}  // namespace

hipError_t launch_quant(const QuantParams& p, hipStream_t stream) {
  const int64_t len = p.transpose ? p.rows : p.cols, lines = p.transpose ? p.cols : p.rows;
  const int64_t n = lines * ((len + 127) / 128) * 4;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (p.type == kTypeF32)
    hipLaunchKernelGGL(quant_kernel<kTypeF32>, grid, dim3(256), 0, stream, p);
  else if (p.type == kTypeBF16)
    hipLaunchKernelGGL(quant_kernel<kTypeBF16>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(quant_kernel<kTypeF16>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_dequant(const DequantParams& p, hipStream_t stream) {
  const int64_t n = p.rows * ((p.cols + 7) / 8);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (p.type == kTypeF32)
    hipLaunchKernelGGL(dequant_kernel<kTypeF32>, grid, dim3(256), 0, stream, p);
  else if (p.type == kTypeBF16)
    hipLaunchKernelGGL(dequant_kernel<kTypeBF16>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(dequant_kernel<kTypeF16>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
