// silu(g) * u of rows X = [g | u], with X kept in e4m3 for the gradient, and the
// gradient from what was kept.
//
//   s = 1 / (1 + exp(-g)),  y = g s u
//   dg = dy u s (1 + g (1 - s)),  du = dy g s
//
// One pass each, row by row, bound by memory: 32768 x 2048 bf16 to e4m3 and back, both
// with everything quantised, 876 MB in 164 to 173 us (5.1 to 5.3 TB/s).  Four rows to a wave:
// two 172 us, eight 184.
#include "common.hpp"
#include "fp8_rows.hpp"

namespace pgk {
namespace {

// 1 / (1 + exp(-g)) with an exponential that cannot overflow: of a large one the
// reciprocal is zero where the value is not (g below -87.3).
__device__ __forceinline__ float sigmoid(float g) {
  const float t = expf(-fabsf(g));
  return __builtin_amdgcn_rcpf(1.0f + t) * (g < 0.0f ? t : 1.0f);
}

__device__ __forceinline__ int64_t used_rows(const int* valid, int64_t rows) {
  if (!valid) return rows;
  const int64_t n = *valid;
  return n < 0 ? 0 : n < rows ? n : rows;
}

template <int T, int RW, bool QUANT, bool NT>
__global__ void __launch_bounds__(kRowThreads) glu_kernel(GluParams p) {
  constexpr int ROWS = 4 * RW;
  __shared__ TileScales<RW> s_y, s_g, s_u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t used = used_rows(p.valid, p.rows);
  const int64_t kp = (p.cols + 127) / 128 * 128, ctiles = (p.cols + kRowCols - 1) / kRowCols;
  const int64_t tiles = (used + ROWS - 1) / ROWS * ctiles;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t row0 = rt * ROWS + wave * RW, c = ct * kRowCols + lane * 8;
    Vec8<T> g[RW], u[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const char* x = static_cast<const char*>(p.X) + (row0 + r < used ? row0 + r : used - 1) * p.ldx * size_of(T);
      g[r] = vec8_load<T, false, NT>(x, c, p.cols);
      u[r] = vec8_load<T, false, NT>(x + p.cols * size_of(T), c, p.cols);
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r;
      const bool on = row < used && c < kp;
      float a[8], b[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = vec8_get(g[r], e);
        b[e] = vec8_get(u[r], e);
        y[e] = a[e] * sigmoid(a[e]) * b[e];
      }
      if (p.kept) {
        unsigned byte;
        uint8_t* k = p.kept + row * 2 * kp + c;
        const u32x2_d qg = e4m3_codes(a, byte);
        s_g.put(lane, wave * RW + r, byte);
        const u32x2_d qu = e4m3_codes(b, byte);
        s_u.put(lane, wave * RW + r, byte);
        if (on) {
          *reinterpret_cast<u32x2_d*>(k) = qg;
          *reinterpret_cast<u32x2_d*>(k + kp) = qu;
        }
      }
      if (QUANT) {
        unsigned byte;
        const u32x2_d q = e4m3_codes(y, byte);
        s_y.put(lane, wave * RW + r, byte);
        if (on) *reinterpret_cast<u32x2_d*>(static_cast<uint8_t*>(p.Y) + row * kp + c) = q;
      } else if (row < used) {
        vec8_store<T>(static_cast<char*>(p.Y) + row * p.ldy * size_of(T), c, p.cols, vec8_pack<T>(y));
      }
    }
    if (QUANT || p.kept) {
      __syncthreads();
      if (QUANT) s_y.store(p.y_scale, ct * 4, kp / 128, rt * ROWS, used, p.rows);
      if (p.kept) {
        s_g.store(p.kept_scale, ct * 4, kp / 128, rt * ROWS, used, p.rows);
        s_u.store(p.kept_scale + kp / 128 * p.rows, ct * 4, kp / 128, rt * ROWS, used, p.rows);
      }
      __syncthreads();
    }
  }
}

// KEPT: X is what the forward kept; otherwise the rows themselves.
template <int T, int RW, bool KEPT, bool QUANT, bool NT>
__global__ void __launch_bounds__(kRowThreads) glu_grad_kernel(GluGradParams p) {
  constexpr int ROWS = 4 * RW;
  __shared__ TileScales<RW> s_g, s_u;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t used = used_rows(p.valid, p.rows);
  const int64_t kp = (p.cols + 127) / 128 * 128, ctiles = (p.cols + kRowCols - 1) / kRowCols;
  const int64_t tiles = (used + ROWS - 1) / ROWS * ctiles;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t row0 = rt * ROWS + wave * RW, c = ct * kRowCols + lane * 8;
    Vec8<T> d[RW], g[KEPT ? 1 : RW], u[KEPT ? 1 : RW];
    u32x2_d qg[RW], qu[RW];
    unsigned bg[RW], bu[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r < used ? row0 + r : used - 1;
      d[r] = vec8_load<T, false, NT>(static_cast<const char*>(p.dY) + row * p.ldy * size_of(T), c, p.cols);
      if (KEPT) {
        const int64_t at = c < kp ? c : 0;  // columns past the row: any codes
        const uint8_t* k = static_cast<const uint8_t*>(p.X) + row * 2 * kp + at;
        qg[r] = *reinterpret_cast<const u32x2_d*>(k);
        qu[r] = *reinterpret_cast<const u32x2_d*>(k + kp);
        bg[r] = p.x_scale[(at >> 7) * p.rows + row];
        bu[r] = p.x_scale[((at + kp) >> 7) * p.rows + row];
      } else {
        const char* x = static_cast<const char*>(p.X) + row * p.ldx * size_of(T);
        g[r] = vec8_load<T>(x, c, p.cols);
        u[r] = vec8_load<T>(x + p.cols * size_of(T), c, p.cols);
      }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r;
      const bool on = row < used && c < kp;
      float a[8], b[8];
      if (KEPT) {
        e4m3_values(qg[r], bg[r], a);
        e4m3_values(qu[r], bu[r], b);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = vec8_get(g[r], e);
          b[e] = vec8_get(u[r], e);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dy = vec8_get(d[r], e), s = sigmoid(a[e]), gs = a[e] * s;
        const float dg = dy * b[e] * __builtin_fmaf(gs, 1.0f - s, s);
        b[e] = dy * gs;
        a[e] = dg;
      }
      if (QUANT) {
        unsigned byte;
        uint8_t* q = static_cast<uint8_t*>(p.dX) + row * 2 * kp + c;
        const u32x2_d og = e4m3_codes(a, byte);
        s_g.put(lane, wave * RW + r, byte);
        const u32x2_d ou = e4m3_codes(b, byte);
        s_u.put(lane, wave * RW + r, byte);
        if (on) {
          *reinterpret_cast<u32x2_d*>(q) = og;
          *reinterpret_cast<u32x2_d*>(q + kp) = ou;
        }
      } else if (row < used) {
        char* x = static_cast<char*>(p.dX) + row * p.lddx * size_of(T);
        vec8_store<T>(x, c, p.cols, vec8_pack<T>(a));
        vec8_store<T>(x + p.cols * size_of(T), c, p.cols, vec8_pack<T>(b));
      }
    }
    if (QUANT) {
      __syncthreads();
      s_g.store(p.dx_scale, ct * 4, kp / 128, rt * ROWS, used, p.rows);
      s_u.store(p.dx_scale + kp / 128 * p.rows, ct * 4, kp / 128, rt * ROWS, used, p.rows);
      __syncthreads();
    }
  }
}

constexpr int kTall = 4;  // rows per wave where the tiles fill the device
constexpr int64_t kPastCaches = 128ll << 20;

template <int T, int RW, bool NT>
void glu_sized(const GluParams& p, hipStream_t stream) {
  const dim3 grid = row_grid(row_tiles(p.rows, p.cols, RW));
  if (p.y_scale)
    hipLaunchKernelGGL((glu_kernel<T, RW, true, NT>), grid, dim3(kRowThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((glu_kernel<T, RW, false, NT>), grid, dim3(kRowThreads), 0, stream, p);
}

template <int T, int RW, bool NT>
void glu_grad_sized(const GluGradParams& p, hipStream_t stream) {
  const dim3 grid = row_grid(row_tiles(p.rows, p.cols, RW)), block(kRowThreads);
  if (p.x_scale) {
    if (p.dx_scale)
      hipLaunchKernelGGL((glu_grad_kernel<T, RW, true, true, NT>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((glu_grad_kernel<T, RW, true, false, NT>), grid, block, 0, stream, p);
  } else {
    if (p.dx_scale)
      hipLaunchKernelGGL((glu_grad_kernel<T, RW, false, true, NT>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((glu_grad_kernel<T, RW, false, false, NT>), grid, block, 0, stream, p);
  }
}

// Inputs that fill most of the Infinity Cache are loaded past the caches where a load
// covers whole lines: 16 bits, rows (and u's half of X) that start on them.  Smaller ones are
// not, behind the product that made them, 16 MB, both calls, 27.0 / 27.3 (but 64 MB 64.5 /
// 71.3, 128 MB 128 / 128).  us, past the caches / through them.  32768 x 2048
// bf16: forward 92.7 / 93.3, backward from X 119 / 122, to e4m3 87 / 87 to 90; 17000 rows
// forward 48.2 / 50.3; 8192 x 8192 forward, rows not quantised, 94.6 / 96.9, backward 92.4 /
// 94.4.  Rows on 16 bytes only, 2040 columns: forward 127 / 121, without what is kept 100 /
// 97.8; rows that start anywhere, 2047 columns, 231 / 216 and 204 / 189 (backward level).
// fp32, of which a load covers half of each line, 16384 x 2048: forward 95 / 90 and 81 / 76,
// backward 106 / 103; 2047 columns 123 / 112 and 106 / 98.
template <int T>
bool past_caches(const void* x, int64_t ld, int64_t rows, int64_t cols) {
  return rows * cols * size_of(T) >= kPastCaches && rows_at(x, ld, size_of(T), 128);
}

template <int T>
void glu_typed(const GluParams& p, hipStream_t stream) {
  if (row_tiles(p.rows, p.cols, kTall) < 2 * p.cus) {
    glu_sized<T, 1, false>(p, stream);
    return;
  }
  if constexpr (T != kTypeF32) {
    if (past_caches<T>(p.X, p.ldx, p.rows, 2 * p.cols) && p.cols * size_of(T) % 128 == 0) {
      glu_sized<T, kTall, true>(p, stream);
      return;
    }
  }
  glu_sized<T, kTall, false>(p, stream);
}
template <int T>
void glu_grad_typed(const GluGradParams& p, hipStream_t stream) {
  if (row_tiles(p.rows, p.cols, kTall) < 2 * p.cus) {
    glu_grad_sized<T, 1, false>(p, stream);
    return;
  }
  if constexpr (T != kTypeF32) {
    if (past_caches<T>(p.dY, p.ldy, p.rows, p.cols)) {
      glu_grad_sized<T, kTall, true>(p, stream);
      return;
    }
  }
  glu_grad_sized<T, kTall, false>(p, stream);
}

}  // namespace

hipError_t launch_glu(const GluParams& p, hipStream_t stream) {
  if (p.type == kTypeF32)
    glu_typed<kTypeF32>(p, stream);
  else if (p.type == kTypeBF16)
    glu_typed<kTypeBF16>(p, stream);
  else
    glu_typed<kTypeF16>(p, stream);
  return hipGetLastError();
}

hipError_t launch_glu_grad(const GluGradParams& p, hipStream_t stream) {
  if (p.type == kTypeF32)
    glu_grad_typed<kTypeF32>(p, stream);
  else if (p.type == kTypeBF16)
    glu_grad_typed<kTypeBF16>(p, stream);
  else
    glu_grad_typed<kTypeF16>(p, stream);
  return hipGetLastError();
}

}  // namespace pgk
