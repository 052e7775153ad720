// What the norm's kernels and its gradient's share: how the threads of a
// workgroup divide a row, and the sums over them.
//
// A row is cut into vectors of eight columns, VPT of them per thread (vector i
// of thread t starts at column 8 * (i * L + t), so a wave's load is one
// consecutive stretch).  L threads hold a row: 16, 32 or 64 lanes of a wave
// for short rows, a workgroup of 256 then taking 256 / L rows; whole waves,
// and one row per workgroup, for longer ones.
#pragma once

#include "mx_device.hpp"

namespace pgk {

constexpr int kRmsMaxLanes = 1024;

struct RmsShape {
  int lanes;    // L
  int threads;  // of a workgroup
  int rows;     // rows a workgroup takes at once
};

// Threads for rows of kp columns (a multiple of 128) at vpt vectors each.
inline RmsShape rms_shape(int64_t kp, int vpt) {
  const int64_t need = (kp / 8 + vpt - 1) / vpt;
  if (need > 64) {
    const int l = (int)((need + 63) / 64 * 64);
    return {l, l, 1};
  }
  const int l = need <= 16 ? 16 : need <= 32 ? 32 : 64;
  return {l, 256, 256 / l};
}

// Sum over the L threads of each row, in all of them.  `s`: 2 * 16 elements of
// LDS; the two halves take turns (`turn`), so that one barrier per call is
// enough.  Every thread of the workgroup calls it.
template <class T>
__device__ __forceinline__ T row_sum(T v, int L, T (*s)[16], int turn) {
  for (int d = L < 64 ? L / 2 : 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if (L <= 64) return v;
  const int waves = L >> 6;
  if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[turn][0];
  for (int w = 1; w < waves; ++w) v += s[turn][w];
  return v;
}

// A vector of a type known at run time (the same for all threads) as fp32.
template <int T>
__device__ __forceinline__ void vec8_f32(const Vec8<T>& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = vec8_get(v, e);
}

}  // namespace pgk
