// What the norm's kernels and its gradient's share: how the threads of a
// workgroup divide a row, and the sums over them.
//
// A row is cut into vectors of eight columns, VPT of them per thread (vector i
// of thread t starts at column 8 * (i * L + t), so a wave's load is one
// consecutive stretch).  L threads hold a row: 16 or 32 lanes of a wave, or
// whole waves; a workgroup takes as many rows side by side as it has room for.
#pragma once

#include "mx_device.hpp"

namespace pgk {

constexpr int kRmsMaxLanes = 1024;

// Threads L for rows of kp columns (a multiple of 128) at vpt vectors each.
inline int rms_lanes(int64_t kp, int vpt) {
  const int64_t need = (kp / 8 + vpt - 1) / vpt;
  return need <= 16 ? 16 : need <= 32 ? 32 : (int)((need + 63) / 64 * 64);
}

// The value of a lane's partner, 32 bits at a time: quads and half rows by
// data-parallel primitives, 16 and 32 lanes apart by the row swaps.
template <int CTRL, class T>
__device__ __forceinline__ T dpp(T v) {
  constexpr int n = sizeof(T) / 4;
  int w[n];
  __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
  for (int i = 0; i < n; ++i) w[i] = __builtin_amdgcn_update_dpp(0, w[i], CTRL, 0xf, 0xf, true);
  __builtin_memcpy(&v, w, sizeof(T));
  return v;
}
template <bool HALF, class T>
__device__ __forceinline__ T swap_sum(T v) {
  constexpr int n = sizeof(T) / 4;
  unsigned w[n], a[n], b[n];
  __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const auto r = HALF ? __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false)
                        : __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false);
    a[i] = r[0];
    b[i] = r[1];
  }
  T x, y;
  __builtin_memcpy(&x, a, sizeof(T));
  __builtin_memcpy(&y, b, sizeof(T));
  return x + y;
}

// Sum over the L threads of each row, the same bits in all of them.  `s`: 2 *
// 16 elements of LDS; the two halves take turns (`turn`), so that one barrier
// per call is enough.  Every thread of the workgroup calls it; a row's threads
// start at a multiple of L.
template <class T>
__device__ __forceinline__ T row_sum(T v, int L, T (*s)[16], int turn) {
  v += dpp<0xB1>(v);   // neighbours in a quad
  v += dpp<0x4E>(v);   // pairs in a quad
  v += dpp<0x141>(v);  // mirrored in eight lanes
  v += dpp<0x140>(v);  // mirrored in sixteen
  if (L > 16) v = swap_sum<false>(v);
  if (L > 32) v = swap_sum<true>(v);
  if (L <= 64) return v;
  const int waves = L >> 6, first = (int)threadIdx.x / L * waves;
  if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  v = s[turn][first];
  for (int w = 1; w < waves; ++w) v += s[turn][first + w];
  return v;
}

// A vector of a type known at run time (the same for all threads) as fp32.
template <int T>
__device__ __forceinline__ void vec8_f32(const Vec8<T>& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = vec8_get(v, e);
}

}  // namespace pgk
