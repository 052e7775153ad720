// Root-mean-square norm of rows with the residual's addition before it and
// the quantisation of the next product's operand after it.
//
// One pass over the data: a row's h = x + r stays in registers between the sum
// of squares and the output, and its blocks' scale exponents are found there
// too.  Bound by memory (8192 x 8192 bf16 with residual to e4m3: 470 MB in 84 to
// 98 us, 4.8 to 5.6 TB/s, the first hundred calls of a run the slowest, where a
// copy of that size reaches 5.2); the arithmetic is in 64 bits (which gfx950 runs
// at the rate of unpacked 32-bit operations), because the quantised outputs round
// at borders: y in fp32 would now and then be on the other side of one, and a
// scale byte off by one is a factor of two.
#include "common.hpp"
#include "rms_device.hpp"

namespace pgk {
namespace {

// y in 64 bits, as fp32 with the bits below the 20th of the fraction folded
// into the last one (round to odd): whatever few bits the result is rounded to
// next, it is rounded as from the 64-bit value.  (Below 2^-126 fp32 itself has
// fewer bits, and the result may be rounded twice.)
__device__ __forceinline__ float narrow_odd(double y) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, y);
  const unsigned lo = (unsigned)b, hi = (unsigned)(b >> 32);
  return (float)__builtin_bit_cast(double, (unsigned long long)(hi | (lo != 0u ? 1u : 0u)) << 32);
}

// How the rows are divided: L threads to a row, `per` rows side by side in a
// workgroup, n groups of them.
struct RowPlan {
  int L, per;
  unsigned n;
  unsigned full;  // groups in whole rounds of xcds << shift
  unsigned xcds;
  int shift;
};

// The row group of workgroup i: ranges of 2^shift consecutive ones go to the
// workgroups of one XCD (which take every xcds-th index), because the scale bytes
// of consecutive rows share lines of memory, which that XCD's L2 then writes
// whole.  (32 bits and one division: every workgroup computes it before its
// first load.)
__device__ __forceinline__ unsigned group_of(unsigned i, const RowPlan& g) {
  if (i >= g.full) return i;
  const unsigned j = i / g.xcds, x = i - j * g.xcds;
  return ((((j >> g.shift) * g.xcds) + x) << g.shift) + (j & ((1u << g.shift) - 1u));
}

// 1 / sqrt(x) to the last bit or two: the approximate instruction and two
// Newton steps, a third of the instructions of a square root and a division,
// which every wave of a row would run.  Zero and infinity as the instruction
// has them.
__device__ __forceinline__ double inv_sqrt(double x) {
  const double r0 = __builtin_amdgcn_rsq(x);
  double r = r0;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = r + r * (0.5 - 0.5 * x * r * r);
  return x > 0.0 && x < __builtin_inf() ? r : r0;
}

template <int WT, bool WHOLE>
__device__ __forceinline__ void weights(const RmsParams& p, int64_t c, float (&w)[8]) {
  vec8_f32<WT>(vec8_load<WT, WHOLE>(p.W, c, p.cols), w);
}

// h = x + r as it is stored (RT: its type), written to H where there is a
// residual.
template <int XT, int RT, bool RES, bool WHOLE, bool STREAM>
__device__ __forceinline__ void h_of(const RmsParams& p, int64_t row, int64_t c, const Vec8<XT>& x, const Vec8<RT>& r,
                                     float (&h)[8]) {
  vec8_f32<XT>(x, h);
  if (RES) {
    float a[8];
    vec8_f32<RT>(r, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] += h[e];
    const Vec8<RT> s = vec8_pack<RT>(a);
    vec8_store<RT, WHOLE, STREAM && WHOLE>(static_cast<char*>(p.H) + row * p.ldh * (RT == kTypeF32 ? 4 : 2), c, p.cols, s);
    vec8_f32<RT>(s, h);
  }
}

// Eight columns of the output.  Called by whole rows of 16 lanes.
template <int XT, int OUT, bool WHOLE>
__device__ __forceinline__ void put(const RmsParams& p, int64_t row, int64_t c, int64_t kp, const float (&h)[8],
                                    const float (&w)[8], double rstd) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double v = (double)h[e] * (double)w[e] * rstd;
    y[e] = OUT == kRmsSame && XT == kTypeF32 ? (float)v : narrow_odd(v);
  }
  if (OUT == kRmsSame) {
    vec8_store<XT, WHOLE>(static_cast<char*>(p.Y) + row * p.ldy * (XT == kTypeF32 ? 4 : 2), c, p.cols, vec8_pack<XT>(y));
    return;
  }
  if (!WHOLE && c + 8 > p.cols) {  // the padding is zero whatever rstd is
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= p.cols) y[e] = 0.0f;
  }
  if (WHOLE && c >= p.cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
  }
  const Vec8<kTypeF32> v = vec8_pack<kTypeF32>(y);
  const int lane16 = threadIdx.x & 15;
  uint8_t* q = static_cast<uint8_t*>(p.Y);
  if (OUT == kRmsFp8) {
    const unsigned byte = scale_byte<E4M3>(row16_max(vec8_amax(v)), kRuleCeil);
    const float sc = scale_value(byte);
    u32x2_d o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s16x2_d t = {0, 0};
      t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, y[4 * i], y[4 * i + 1], sc, false);
      t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, y[4 * i + 2], y[4 * i + 3], sc, true);
      o[i] = byte == 255u ? 0u : __builtin_bit_cast(unsigned, t);
    }
    *reinterpret_cast<u32x2_d*>(q + row * kp + c) = o;
    if (lane16 == 0) p.y_scale[(c >> 7) * p.rows + row] = (uint8_t)byte;
  } else {
    const unsigned byte = scale_byte<E2M1>(quad_max(vec8_amax(v)), kRuleCeil);
    const unsigned o = vec8_e2m1(v, scale_value(byte));
    *reinterpret_cast<unsigned*>(q + row * (kp >> 1) + (c >> 1)) = byte == 255u ? 0u : o;
    // the bytes of the row's four blocks of 32 as one word
    unsigned word = byte << (8 * (lane16 >> 2));
    word |= (unsigned)__builtin_amdgcn_update_dpp(0, (int)word, 0x124, 0xf, 0xf, true);
    word |= (unsigned)__builtin_amdgcn_update_dpp(0, (int)word, 0x128, 0xf, 0xf, true);
    if (lane16 == 0) reinterpret_cast<unsigned*>(p.y_scale)[(c >> 7) * p.rows + row] = word;
  }
}

// Rows held in registers: VPT vectors per thread.
template <int XT, int RT, bool RES, int OUT, int VPT, bool WHOLE>
__global__ void __launch_bounds__(VPT == 1 ? kRmsMaxLanes : kRmsMaxLanes / 2) rms_kernel(RmsParams p, RowPlan g) {
  __shared__ double s_sum[2][16];
  const int L = g.L, sub = (int)threadIdx.x / L, t0 = (int)threadIdx.x - sub * L;
  const int64_t kp = (p.cols + 127) / 128 * 128;
  constexpr int xsz = XT == kTypeF32 ? 4 : 2, rsz = RT == kTypeF32 ? 4 : 2;
  // Rows that fill the device pass through the caches once: inputs of 16 bits and
  // h non-temporal (8192 x 8192 bf16 to e4m3 98 -> 94 us, h alone 97, to bf16 101 ->
  // 88; 4864 x 8000 with r in fp32 107 -> 99 by h alone, 104 with r's loads too; 4096
  // x 2056 20.0 -> 17.3, 2048 x 2048 level; rows at odd offsets, whose h stays in the
  // caches, level: 8192 x 8191 152 -> 154).  A reader of h that follows at once, the
  // next norm's residual, loses part of that on small tensors: two norms in a row
  // 1024 x 4096 15.6 -> 16.8 us, 4096 x 4096 49 both ways, 8192 x 8192 175 -> 167.  y
  // stays for its product.
  constexpr bool STREAM = VPT == 4;
  int turn = 0;
  for (unsigned i = blockIdx.x; i < g.n; i += gridDim.x, turn ^= 1) {
    const int64_t row = (int64_t)group_of(i, g) * g.per + sub;
    const bool on = row < p.rows;
    const int64_t at = on ? row : p.rows - 1;
    Vec8<XT> x[VPT];
    Vec8<RT> r[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int64_t c = ((int64_t)v * L + t0) * 8;
      x[v] = vec8_load<XT, WHOLE, STREAM && XT != kTypeF32>(static_cast<const char*>(p.X) + at * p.ldx * xsz, c, p.cols);
      if (RES) r[v] = vec8_load<RT, WHOLE, STREAM && RT != kTypeF32>(static_cast<const char*>(p.R) + at * p.ldr * rsz, c, p.cols);
    }
    float h[VPT][8];
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int64_t c = ((int64_t)v * L + t0) * 8;
      h_of<XT, RT, RES, WHOLE, STREAM>(p, at, on ? c : p.cols, x[v], r[v], h[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (double)h[v][e] * (double)h[v][e];
    }
    s = row_sum(s, L, s_sum, turn);
    const double rstd = inv_sqrt(s * p.inv_cols + p.eps);
    if (!on) continue;
    if (t0 == 0 && p.rstd) p.rstd[row] = (float)rstd;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int64_t c = ((int64_t)v * L + t0) * 8;
      if (c >= kp) continue;
      float w[8];
      if (p.w_type == kTypeF32)
        weights<kTypeF32, WHOLE>(p, c, w);
      else
        weights<XT, WHOLE>(p, c, w);
      put<XT, OUT, WHOLE>(p, row, c, kp, h[v], w, rstd);
    }
  }
}

// Rows too long for that: a workgroup walks the row twice, the second time
// from h as stored.
template <int XT, int RT, bool RES, int OUT>
__global__ void __launch_bounds__(kRmsMaxLanes) rms_long_kernel(RmsParams p) {
  __shared__ double s_sum[2][16];
  const int64_t kp = (p.cols + 127) / 128 * 128;
  constexpr int xsz = XT == kTypeF32 ? 4 : 2, rsz = RT == kTypeF32 ? 4 : 2;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const char* xr = static_cast<const char*>(p.X) + row * p.ldx * xsz;
    double s = 0.0;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += kRmsMaxLanes * 8) {
      Vec8<RT> r;
      if (RES) r = vec8_load<RT>(static_cast<const char*>(p.R) + row * p.ldr * rsz, c, p.cols);
      float h[8];
      h_of<XT, RT, RES, false, false>(p, row, c, vec8_load<XT>(xr, c, p.cols), r, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += (double)h[e] * (double)h[e];
    }
    s = row_sum(s, kRmsMaxLanes, s_sum, turn);
    const double rstd = inv_sqrt(s * p.inv_cols + p.eps);
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = (float)rstd;
    for (int64_t c = threadIdx.x * 8; c < kp; c += kRmsMaxLanes * 8) {
      float h[8], w[8];
      if (RES)  // this thread's own stores
        vec8_f32<RT>(vec8_load<RT>(static_cast<const char*>(p.H) + row * p.ldh * rsz, c, p.cols), h);
      else
        vec8_f32<XT>(vec8_load<XT>(xr, c, p.cols), h);
      if (p.w_type == kTypeF32)
        weights<kTypeF32, false>(p, c, w);
      else
        weights<XT, false>(p, c, w);
      put<XT, OUT, false>(p, row, c, kp, h, w, rstd);
    }
  }
}

constexpr int64_t kMaxGrid = 1 << 20;  // a grid's threads have to stay below 2^32

template <int XT, int RT, bool RES, int OUT>
void launch_typed(const RmsParams& p, hipStream_t stream) {
  const int64_t kp = (p.cols + 127) / 128 * 128;
  // rows whose scale bytes fill a 128-byte line
  const int line = p.out == kRmsFp8 ? 128 : p.out == kRmsFp4 ? 32 : 1;
  // A row's reduction and its 1 / sqrt are work per wave, so few waves per row
  // where rows fill the device; for a handful, as many as there are.
  const int vpt = p.rows <= p.cus && kp <= 8 * kRmsMaxLanes ? 1 : 4;
  if (kp > 16384) {
    const unsigned g = (unsigned)(p.rows < kMaxGrid ? p.rows : kMaxGrid);
    hipLaunchKernelGGL((rms_long_kernel<XT, RT, RES, OUT>), dim3(g), dim3(kRmsMaxLanes), 0, stream, p);
    return;
  }
  const int L = rms_lanes(kp, vpt), per = L < 256 ? 256 / L : 1;
  const dim3 threads(L * per);
  const int64_t n = (p.rows + per - 1) / per;
  const dim3 grid((unsigned)(n < kMaxGrid ? n : kMaxGrid));
  RowPlan g = {L, per, (unsigned)n, 0, (unsigned)p.xcds, 0};
  while ((per << g.shift) < line) ++g.shift;
  g.full = (unsigned)(n / ((int64_t)p.xcds << g.shift) * ((int64_t)p.xcds << g.shift));
  const bool whole = p.cols % 8 == 0;
  if (vpt == 1 && whole)
    hipLaunchKernelGGL((rms_kernel<XT, RT, RES, OUT, 1, true>), grid, threads, 0, stream, p, g);
  else if (vpt == 1)
    hipLaunchKernelGGL((rms_kernel<XT, RT, RES, OUT, 1, false>), grid, threads, 0, stream, p, g);
  else if (whole)
    hipLaunchKernelGGL((rms_kernel<XT, RT, RES, OUT, 4, true>), grid, threads, 0, stream, p, g);
  else
    hipLaunchKernelGGL((rms_kernel<XT, RT, RES, OUT, 4, false>), grid, threads, 0, stream, p, g);
}

template <int XT, int RT, bool RES>
void launch_out(const RmsParams& p, hipStream_t stream) {
  if (p.out == kRmsSame)
    launch_typed<XT, RT, RES, kRmsSame>(p, stream);
  else if (p.out == kRmsFp8)
    launch_typed<XT, RT, RES, kRmsFp8>(p, stream);
  else
    launch_typed<XT, RT, RES, kRmsFp4>(p, stream);
}

template <int XT>
void launch_res(const RmsParams& p, hipStream_t stream) {
  if (!p.R)
    launch_out<XT, XT, false>(p, stream);
  else if (XT == kTypeF32 || p.r_type != kTypeF32)
    launch_out<XT, XT, true>(p, stream);
  else
    launch_out<XT, kTypeF32, true>(p, stream);
}

}  // namespace

hipError_t launch_rms(const RmsParams& p, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  if (p.x_type == kTypeF32)
    launch_res<kTypeF32>(p, stream);
  else if (p.x_type == kTypeBF16)
    launch_res<kTypeBF16>(p, stream);
  else
    launch_res<kTypeF16>(p, stream);
  return hipGetLastError();
}

}  // namespace pgk
