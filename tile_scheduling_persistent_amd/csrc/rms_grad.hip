// Gradient of the RMS norm:
//   g = w * dy, n = h * rstd, dx = dh + rstd * (g - n * mean(g * n))
//   dw = sum over the rows of dy * n
// n is of order one whatever h's size is, so no power of rstd or sum of h
// leaves the range of fp32 before the result does.
//
// One pass over dy, h and dh gives both.  A workgroup walks a strided set of
// rows; its threads own columns, so their shares of dw stay in registers
// (fp32) over the whole walk and leave once, as one row of partial sums.  The
// next row's loads go out before this row's sum is waited for.  A second
// kernel adds the partial sums in a fixed order: results repeat bit for bit.
// Bound by memory: 8192 x 8192 bf16 with dh, 537 MB, in 100 to 105 us, 5.1 to 5.4
// TB/s, a copy's rate.  One workgroup per CU: more of them leave more partial
// sums than they hide.
#include "common.hpp"
#include "rms_device.hpp"

namespace pgk {
namespace {

constexpr int kThreads = 256;

template <int YT, int HT, int VPT>
struct GradRow {
  Vec8<YT> dy[VPT];
  Vec8<HT> h[VPT], dh[VPT];
  float rstd;
};

// The inputs' last use: NT, those of 16 bits non-temporal, where their rows
// start on 16 bytes (8192 x 8192 bf16 103.4 -> 98.4 us, with fp32 h 172.8 -> 166.3;
// dx stored that way too costs 2 us).  Not where lines are shared by two loads,
// which then fetch them twice: 8192 x 8191 bf16 215 -> 234; 8192 x 8192 all in fp32,
// whose loads cover half of each line, 198 -> 209.
template <bool NT, int YT, int HT, int VPT>
__device__ __forceinline__ void load_row(const RmsGradParams& p, int64_t row, int L, int t0,
                                         GradRow<YT, HT, VPT>& g) {
  constexpr int ysz = YT == kTypeF32 ? 4 : 2, hsz = HT == kTypeF32 ? 4 : 2;
  g.rstd = p.rstd[row];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int64_t c = ((int64_t)v * L + t0) * 8;
    g.dy[v] = vec8_load<YT, false, NT && YT != kTypeF32>(static_cast<const char*>(p.dY) + row * p.ldy * ysz, c, p.cols);
    g.h[v] = vec8_load<HT, false, NT && HT != kTypeF32>(static_cast<const char*>(p.H) + row * p.ldh * hsz, c, p.cols);
    if (p.dH) g.dh[v] = vec8_load<HT, false, NT && HT != kTypeF32>(static_cast<const char*>(p.dH) + row * p.ldd * hsz, c, p.cols);
  }
}

template <int YT>
__device__ __forceinline__ void weights(const RmsGradParams& p, int64_t c, float (&w)[8]) {
  if (p.w_type == kTypeF32)
    vec8_f32<kTypeF32>(vec8_load<kTypeF32>(p.W, c, p.cols), w);
  else
    vec8_f32<YT>(vec8_load<YT>(p.W, c, p.cols), w);
}

// dx of eight columns; mean = mean(g * n) of the row.
template <int YT, int HT>
__device__ __forceinline__ void put_dx(const RmsGradParams& p, int64_t row, int64_t c, const float (&dy)[8],
                                       const float (&n)[8], const Vec8<HT>& dh, const float (&w)[8], float rstd,
                                       float mean) {
  float d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    d[e] = rstd * (dy[e] * w[e] - n[e] * mean);
    if (p.dH) d[e] += vec8_get(dh, e);
  }
  vec8_store<HT>(static_cast<char*>(p.dX) + row * p.ldx * (HT == kTypeF32 ? 4 : 2), c, p.cols, vec8_pack<HT>(d));
}

template <int YT, int HT, int VPT, bool AHEAD, bool NT>
__global__ void __launch_bounds__(kRmsMaxLanes) rms_grad_kernel(RmsGradParams p, int L) {
  __shared__ float s_sum[2][16];
  __shared__ float s_dw[VPT == 1 ? kRmsMaxLanes * 8 : 1];
  const int per = (int)blockDim.x / L, sub = (int)threadIdx.x / L, t0 = (int)threadIdx.x - sub * L;
  const int64_t n = (p.rows + per - 1) / per;
  float acc[VPT][8] = {};
  float w[VPT][8];
  auto load_w = [&]() {
#pragma unroll
    for (int v = 0; v < VPT; ++v) weights<YT>(p, ((int64_t)v * L + t0) * 8, w[v]);
  };
  if (VPT == 1) load_w();
  const float inv = 1.0f / (float)p.cols;
  GradRow<YT, HT, VPT> now;
  int64_t i = blockIdx.x;
  auto row_at = [&](int64_t j) {
    const int64_t row = j * per + sub;
    return row < p.rows ? row : p.rows - 1;
  };
  if (AHEAD && i < n) load_row<NT>(p, row_at(i), L, t0, now);
  int turn = 0;
  for (; i < n; i += gridDim.x, turn ^= 1) {
    const bool on = i * per + sub < p.rows;
    const int64_t row = row_at(i);
    GradRow<YT, HT, VPT> next;
    if (AHEAD) {
      if (i + gridDim.x < n) load_row<NT>(p, row_at(i + gridDim.x), L, t0, next);
    } else {
      load_row<NT>(p, row, L, t0, now);
    }
    if (VPT != 1) load_w();  // two vectors leave no registers to keep it in
    const float r = now.rstd;
    float c = 0.0f;
    float dy[VPT][8], nh[VPT][8];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      vec8_f32<YT>(now.dy[v], dy[v]);
      vec8_f32<HT>(now.h[v], nh[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        nh[v][e] *= r;
        c += dy[v][e] * w[v][e] * nh[v][e];
        if (on) acc[v][e] += dy[v][e] * nh[v][e];
      }
    }
    const float mean = row_sum(c, L, s_sum, turn) * inv;
    if (on) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        put_dx<YT, HT>(p, row, ((int64_t)v * L + t0) * 8, dy[v], nh[v], now.dh[v], w[v], r, mean);
    }
    if (AHEAD) now = next;
  }
  if (!p.dW) return;
  if (VPT == 1 && per > 1) {  // the rows the workgroup took side by side
#pragma unroll
    for (int e = 0; e < 8; ++e) s_dw[(sub * L + t0) * 8 + e] = acc[0][e];
    __syncthreads();
    for (int c = threadIdx.x; c < L * 8; c += blockDim.x) {
      float s = 0.0f;
      for (int q = 0; q < per; ++q) s += s_dw[q * L * 8 + c];
      if (c < p.cols) p.ws[(int64_t)blockIdx.x * p.cols + c] = s;
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    vec8_store<kTypeF32>(p.ws + (int64_t)blockIdx.x * p.cols, ((int64_t)v * L + t0) * 8, p.cols,
                         vec8_pack<kTypeF32>(acc[v]));
}

// Rows too long for registers: dw and dx each in a pass of its own, dw first
// because dx may take dy's or dh's place.
template <int YT, int HT>
__global__ void __launch_bounds__(kThreads) rms_grad_long_dw_kernel(RmsGradParams p) {
  constexpr int ysz = YT == kTypeF32 ? 4 : 2, hsz = HT == kTypeF32 ? 4 : 2;
  const int64_t step = (int64_t)gridDim.x * kThreads * 8;
  for (int64_t c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; c < p.cols; c += step) {
    float acc[8] = {};
    for (int64_t row = blockIdx.y; row < p.rows; row += p.partials) {
      float dy[8], h[8];
      vec8_f32<YT>(vec8_load<YT>(static_cast<const char*>(p.dY) + row * p.ldy * ysz, c, p.cols), dy);
      vec8_f32<HT>(vec8_load<HT>(static_cast<const char*>(p.H) + row * p.ldh * hsz, c, p.cols), h);
      const float r = p.rstd[row];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += dy[e] * (h[e] * r);
    }
    vec8_store<kTypeF32>(p.ws + (int64_t)blockIdx.y * p.cols, c, p.cols, vec8_pack<kTypeF32>(acc));
  }
}

template <int YT, int HT>
__global__ void __launch_bounds__(kRmsMaxLanes) rms_grad_long_dx_kernel(RmsGradParams p) {
  __shared__ float s_sum[2][16];
  constexpr int ysz = YT == kTypeF32 ? 4 : 2, hsz = HT == kTypeF32 ? 4 : 2;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const char* yr = static_cast<const char*>(p.dY) + row * p.ldy * ysz;
    const char* hr = static_cast<const char*>(p.H) + row * p.ldh * hsz;
    const float r = p.rstd[row];
    float s = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += kRmsMaxLanes * 8) {
      float dy[8], h[8], w[8];
      vec8_f32<YT>(vec8_load<YT>(yr, c, p.cols), dy);
      vec8_f32<HT>(vec8_load<HT>(hr, c, p.cols), h);
      weights<YT>(p, c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += dy[e] * w[e] * (h[e] * r);
    }
    const float mean = row_sum(s, kRmsMaxLanes, s_sum, turn) / (float)p.cols;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += kRmsMaxLanes * 8) {
      float dy[8], h[8], w[8];
      Vec8<HT> dh;
      vec8_f32<YT>(vec8_load<YT>(yr, c, p.cols), dy);
      vec8_f32<HT>(vec8_load<HT>(hr, c, p.cols), h);
      if (p.dH) dh = vec8_load<HT>(static_cast<const char*>(p.dH) + row * p.ldd * hsz, c, p.cols);
      weights<YT>(p, c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] *= r;
      put_dx<YT, HT>(p, row, c, dy, h, dh, w, r, mean);
    }
  }
}

// dw from the partial sums: 32 columns per workgroup, 32 threads to a column,
// so that the few hundred rows of partial sums are a handful of loads each.
__global__ void __launch_bounds__(1024) rms_dw_sum_kernel(RmsGradParams p) {
  __shared__ float s_part[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < p.cols; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + x;
    float s = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
      for (int q = y; q < p.partials; q += 32) s += p.ws[(int64_t)q * p.cols + c];
    }
    s_part[y][x] = s;
    __syncthreads();
    // eight sums of four, then of two eight times over
    if (y < 8) s_part[y][x] = (s + s_part[y + 8][x]) + (s_part[y + 16][x] + s_part[y + 24][x]);
    __syncthreads();
    if (y == 0 && c < p.cols) {
      for (int q = 1; q < 8; ++q) s_part[0][x] += s_part[q][x];
      p.dW[c] = s_part[0][x];
    }
    __syncthreads();
  }
}

constexpr int kWorkgroupsPerCu = 1;
constexpr int64_t kMaxGrid = 1 << 20;  // a grid's threads have to stay below 2^32

// How the rows are walked.  Up to 8192 columns one vector per thread: a wide
// row keeps 16 waves busy, which leaves each the registers for the next row's
// loads; several shorter rows go side by side in one workgroup, so that the
// partial sums of dw stay one row per workgroup.  Two vectors up to 16384
// columns, then the passes over long rows.
struct GradPlan {
  int vpt;  // 0: long rows
  int lanes, threads, grid;
};
GradPlan grad_plan(int64_t rows, int64_t cols, int cus) {
  const int64_t kp = (cols + 127) / 128 * 128;
  GradPlan g;
  g.vpt = kp <= 8 * kRmsMaxLanes ? 1 : kp <= 16 * kRmsMaxLanes ? 2 : 0;
  if (g.vpt == 0) {
    g.lanes = g.threads = kRmsMaxLanes;
    g.grid = (int)(rows < 64 ? rows : 64);
    return g;
  }
  g.lanes = rms_lanes(kp, g.vpt);
  const int per = g.vpt == 1 ? kRmsMaxLanes / g.lanes : 1;
  g.threads = per * g.lanes;
  const int64_t n = (rows + per - 1) / per;
  g.grid = (int)(n < kWorkgroupsPerCu * cus ? n : kWorkgroupsPerCu * cus);
  return g;
}

template <int YT, int HT, bool NT>
void launch_rows(const RmsGradParams& p, const GradPlan& g, dim3 grid, dim3 threads, hipStream_t stream) {
  if (g.vpt == 1)
    hipLaunchKernelGGL((rms_grad_kernel<YT, HT, 1, true, NT>), grid, threads, 0, stream, p, g.lanes);
  else
    hipLaunchKernelGGL((rms_grad_kernel<YT, HT, 2, false, NT>), grid, threads, 0, stream, p, g.lanes);
}

template <int YT, int HT>
void launch_typed(const RmsGradParams& p, hipStream_t stream) {
  const GradPlan g = grad_plan(p.rows, p.cols, p.cus);
  if (p.rows > 0 && g.vpt == 0) {
    if (p.dW) {
      const int64_t n = (p.cols + kThreads * 8 - 1) / (kThreads * 8);
      const dim3 grid((unsigned)(n < 65536 ? n : 65536), (unsigned)p.partials);
      hipLaunchKernelGGL((rms_grad_long_dw_kernel<YT, HT>), grid, dim3(kThreads), 0, stream, p);
    }
    const unsigned rows = (unsigned)(p.rows < kMaxGrid ? p.rows : kMaxGrid);
    hipLaunchKernelGGL((rms_grad_long_dx_kernel<YT, HT>), dim3(rows), dim3(kRmsMaxLanes), 0, stream, p);
  } else if (p.rows > 0) {
    const dim3 grid((unsigned)(p.dW ? p.partials : g.grid)), threads(g.threads);
    const bool at16 = (YT == kTypeF32 || rows_at(p.dY, p.ldy, 2, 16)) &&
                      (HT == kTypeF32 || (rows_at(p.H, p.ldh, 2, 16) && (!p.dH || rows_at(p.dH, p.ldd, 2, 16))));
    if (YT != kTypeF32 && at16)
      launch_rows<YT, HT, YT != kTypeF32>(p, g, grid, threads, stream);
    else
      launch_rows<YT, HT, false>(p, g, grid, threads, stream);
  }
  if (p.dW) {
    const int64_t n = (p.cols + 31) / 32;
    hipLaunchKernelGGL(rms_dw_sum_kernel, dim3((unsigned)(n < kMaxGrid ? n : kMaxGrid)), dim3(1024), 0, stream, p);
  }
}

}  // namespace

// Rows of partial sums a call leaves (0 rows: none).
int rms_grad_partials(int64_t rows, int64_t cols, int cus) { return grad_plan(rows, cols, cus).grid; }

hipError_t launch_rms_grad(const RmsGradParams& p, hipStream_t stream) {
  if (p.y_type == kTypeF32)
    launch_typed<kTypeF32, kTypeF32>(p, stream);
  else if (p.y_type == kTypeBF16)
    p.h_type == kTypeF32 ? launch_typed<kTypeBF16, kTypeF32>(p, stream) : launch_typed<kTypeBF16, kTypeBF16>(p, stream);
  else
    p.h_type == kTypeF32 ? launch_typed<kTypeF16, kTypeF32>(p, stream) : launch_typed<kTypeF16, kTypeF16>(p, stream);
  return hipGetLastError();
}

}  // namespace pgk
