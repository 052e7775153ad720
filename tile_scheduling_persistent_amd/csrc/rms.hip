// Root-mean-square norm of rows with the residual's addition before it and
// the quantisation of the next product's operand after it, and its gradient.
#include "common.hpp"
#include "mx_device.hpp"

namespace pgk {
namespace {

constexpr int kThreads = 256;

// y = h * rstd * w in 64 bits, as fp32 with the bits below the 20th of the
// fraction folded into the last one (round to odd): whatever few bits the
// result is rounded to next, it is rounded as from the 64-bit value.
__device__ __forceinline__ float narrow_odd(double y) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, y);
  const unsigned lo = (unsigned)b, hi = (unsigned)(b >> 32);
  return (float)__builtin_bit_cast(double, (unsigned long long)(hi | (lo != 0u ? 1u : 0u)) << 32);
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, int type) {
  if (type == kTypeF32) return load_elem<kTypeF32>(p, i);
  if (type == kTypeBF16) return load_elem<kTypeBF16>(p, i);
  return load_elem<kTypeF16>(p, i);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int type, float v) {
  if (type == kTypeF32)
    store_elem<kTypeF32>(p, i, v);
  else if (type == kTypeBF16)
    store_elem<kTypeBF16>(p, i, v);
  else
    store_elem<kTypeF16>(p, i, v);
}

// x rounded to the element type, as fp32.
__device__ __forceinline__ float round_any(float x, int type) {
  if (type == kTypeBF16) return (float)(__bf16)x;
  if (type == kTypeF16) return (float)(_Float16)x;
  return x;
}

template <class T>
__device__ __forceinline__ T block_sum(T v, T* s) {
  const int t = threadIdx.x;
  s[t] = v;
  __syncthreads();
  for (int n = kThreads / 2; n > 0; n >>= 1) {
    if (t < n) s[t] += s[t + n];
    __syncthreads();
  }
  const T r = s[0];
  __syncthreads();
  return r;
}

// One workgroup per row.
__global__ void __launch_bounds__(kThreads) rms_kernel(RmsParams p) {
  __shared__ double red[kThreads];
  const int64_t row = blockIdx.x;
  const int64_t groups = (p.cols + 127) / 128;
  auto h_at = [&](int64_t c) {
    const float x = load_any(p.X, row * p.ldx + c, p.x_type);
    return p.R ? round_any(x + load_any(p.R, row * p.ldr + c, p.r_type), p.r_type) : x;
  };
  double s = 0.0;
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
    const double h = h_at(c);
    s += h * h;
  }
  const double rstd = 1.0 / sqrt(block_sum(s, red) / (double)p.cols + p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[row] = (float)rstd;
  auto y_at = [&](int64_t c, float h) { return (double)h * rstd * (double)load_any(p.W, c, p.w_type); };
  if (p.out == kRmsSame) {
    for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
      const float h = h_at(c);
      const double y = y_at(c, h);
      if (p.H) store_any(p.H, row * p.ldh + c, p.r_type, h);
      store_any(p.Y, row * p.ldy + c, p.x_type, p.x_type == kTypeF32 ? (float)y : narrow_odd(y));
    }
    return;
  }
  const int64_t nblk = p.out == kRmsFp8 ? groups : groups * 4;
  const int len = p.out == kRmsFp8 ? 128 : 32;
  for (int64_t b = threadIdx.x; b < nblk; b += kThreads) {
    unsigned amax = 0;
    for (int e = 0; e < len; ++e) {
      const int64_t c = b * len + e;
      if (c >= p.cols) break;
      const unsigned v = __builtin_bit_cast(unsigned, narrow_odd(y_at(c, h_at(c)))) & 0x7fffffffu;
      amax = v > amax ? v : amax;
    }
    const unsigned byte = p.out == kRmsFp8 ? scale_byte<E4M3>(amax, kRuleCeil) : scale_byte<E2M1>(amax, kRuleCeil);
    const float sc = scale_value(byte);
    for (int e = 0; e < len; e += 8) {
      float y[8];
      for (int i = 0; i < 8; ++i) {
        const int64_t c = b * len + e + i;
        const float h = c < p.cols ? h_at(c) : 0.0f;
        y[i] = c < p.cols && byte != 255u ? narrow_odd(y_at(c, h)) : 0.0f;
        if (p.H && c < p.cols) store_any(p.H, row * p.ldh + c, p.r_type, h);
      }
      if (p.out == kRmsFp8) {
        unsigned* q = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(p.Y) + row * groups * 128 + b * 128 + e);
        for (int i = 0; i < 2; ++i) {
          s16x2_d o = {0, 0};
          o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[4 * i], y[4 * i + 1], sc, false);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[4 * i + 2], y[4 * i + 3], sc, true);
          q[i] = byte == 255u ? 0u : __builtin_bit_cast(unsigned, o);
        }
      } else {
        const unsigned o = vec8_e2m1(vec8_pack<kTypeF32>(y), sc);
        *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(p.Y) + row * groups * 64 + b * 16 + e / 2) =
            byte == 255u ? 0u : o;
      }
    }
    if (p.out == kRmsFp8)
      p.y_scale[b * p.rows + row] = (uint8_t)byte;
    else
      p.y_scale[((b >> 2) * p.rows + row) * 4 + (b & 3)] = (uint8_t)byte;
  }
}

// One workgroup per row: dx.
__global__ void __launch_bounds__(kThreads) rms_dx_kernel(RmsGradParams p) {
  __shared__ float red[kThreads];
  const int64_t row = blockIdx.x;
  const float r = p.rstd[row];
  float s = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads)
    s += load_any(p.dY, row * p.ldy + c, p.y_type) * load_any(p.W, c, p.w_type) * load_any(p.H, row * p.ldh + c, p.h_type);
  const float k = r * r * r * (block_sum(s, red) / (float)p.cols);
  for (int64_t c = threadIdx.x; c < p.cols; c += kThreads) {
    const float g = load_any(p.dY, row * p.ldy + c, p.y_type) * load_any(p.W, c, p.w_type);
    float v = r * g - load_any(p.H, row * p.ldh + c, p.h_type) * k;
    if (p.dH) v += load_any(p.dH, row * p.ldd + c, p.h_type);
    store_any(p.dX, row * p.ldx + c, p.h_type, v);
  }
}

// Partial sums of dw: program q adds the rows q, q + P, ...
__global__ void __launch_bounds__(kThreads) rms_dw_kernel(RmsGradParams p) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += p.partials)
    s += load_any(p.dY, row * p.ldy + c, p.y_type) * (load_any(p.H, row * p.ldh + c, p.h_type) * p.rstd[row]);
  p.ws[(int64_t)blockIdx.y * p.cols + c] = s;
}

__global__ void __launch_bounds__(kThreads) rms_dw_sum_kernel(RmsGradParams p) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  float s = 0.0f;
  for (int q = 0; q < p.partials; ++q) s += p.ws[(int64_t)q * p.cols + c];
  p.dW[c] = s;
}

}  // namespace

hipError_t launch_rms(const RmsParams& p, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  hipLaunchKernelGGL(rms_kernel, dim3((unsigned)p.rows), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

int rms_grad_partials(int64_t rows) { return (int)(rows < 64 ? rows : 64); }

hipError_t launch_rms_grad(const RmsGradParams& p, hipStream_t stream) {
  const unsigned cb = (unsigned)((p.cols + kThreads - 1) / kThreads);
  if (p.dW) {  // before dX, which may take dY's place
    if (p.partials > 0) hipLaunchKernelGGL(rms_dw_kernel, dim3(cb, (unsigned)p.partials), dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL(rms_dw_sum_kernel, dim3(cb), dim3(kThreads), 0, stream, p);
  }
  if (p.rows > 0) hipLaunchKernelGGL(rms_dx_kernel, dim3((unsigned)p.rows), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace pgk
