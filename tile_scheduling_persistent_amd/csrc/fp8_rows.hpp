// e4m3 with one e8m0 scale per 128 consecutive columns of a row, eight columns
// per lane: what the kernels that make or read such rows share.
#pragma once

#include "mx_device.hpp"

namespace pgk {

// Codes of a lane's eight values and the scale byte of its block, which the 16
// lanes of its row of lanes share (all of them call).
__device__ __forceinline__ u32x2_d e4m3_codes(const float (&y)[8], unsigned& byte) {
  byte = scale_byte<E4M3>(row16_max(vec8_amax(vec8_pack<kTypeF32>(y))), kRuleCeil);
  const float sc = scale_value(byte);
  u32x2_d o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s16x2_d t = {0, 0};
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, y[4 * i], y[4 * i + 1], sc, false);
    t = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(t, y[4 * i + 2], y[4 * i + 3], sc, true);
    o[i] = byte == 255u ? 0u : __builtin_bit_cast(unsigned, t);
  }
  return o;
}

// The values of eight codes under scale byte `byte` (exact down to 2^-149).
__device__ __forceinline__ void e4m3_values(u32x2_d codes, unsigned byte, float (&x)[8]) {
  const float sc = scale_value(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned w = i == 0 ? codes[0] : codes[1];  // the element first: a builtin's argument takes no vector element
    const f32x2_d a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[4 * i] = a[0] * sc;
    x[4 * i + 1] = a[1] * sc;
    x[4 * i + 2] = b[0] * sc;
    x[4 * i + 3] = b[1] * sc;
  }
}

// A tile of the kernels that work row by row: 4 * RW rows of 512 columns, RW
// rows to a wave, eight columns (one vector, 16 bytes of 16-bit elements) to a
// lane, all loads of a wave in flight before the first is used.
constexpr int kRowThreads = 256;
constexpr int kRowCols = 512;
// Workgroups a launch has at most; past them each takes several tiles (a grid's
// threads have to stay below 2^32).
constexpr int64_t kRowGrid = 1 << 20;

// The scale bytes of a tile, collected in LDS: in memory a group's bytes of
// consecutive rows stand side by side.
template <int RW>
struct TileScales {
  unsigned char b[4][4 * RW];
  // By the lane that holds the first vector of a block.
  __device__ __forceinline__ void put(int lane, int row, unsigned byte) {
    if ((lane & 15) == 0) b[lane >> 4][row] = (unsigned char)byte;
  }
  // By every thread, between two barriers: groups g0 .. (below `groups`) of rows
  // row0 .. (below `rows`) into scale [groups][ld].
  __device__ __forceinline__ void store(uint8_t* scale, int64_t g0, int64_t groups, int64_t row0, int64_t rows,
                                        int64_t ld) const {
    for (int i = threadIdx.x; i < 16 * RW; i += kRowThreads) {
      const int64_t g = g0 + i / (4 * RW), row = row0 + i % (4 * RW);
      if (g < groups && row < rows) scale[g * ld + row] = b[i / (4 * RW)][i % (4 * RW)];
    }
  }
};

inline dim3 row_grid(int64_t tiles) { return dim3((unsigned)(tiles < kRowGrid ? tiles : kRowGrid)); }
inline int64_t row_tiles(int64_t rows, int64_t cols, int rw) {
  return (rows + 4 * rw - 1) / (4 * rw) * ((cols + kRowCols - 1) / kRowCols);
}

constexpr int size_of(int type) { return type == kTypeF32 ? 4 : 2; }

}  // namespace pgk
