// The rows and output tiles of experts, from the offsets in device memory.
#pragma once

#include "common.hpp"

namespace pgk {

// Rows [lo, lo + n) of an expert.  Offsets outside of [0, rows], or that fall,
// give an empty or shorter range, never one past the rows.
struct ExpertRows {
  int lo, n;
};
__device__ __forceinline__ ExpertRows expert_rows(const int* offsets, int e, int rows) {
  if (!offsets) return {0, rows};
  int lo = offsets[e], hi = offsets[e + 1];
  lo = lo < 0 ? 0 : lo < rows ? lo : rows;
  hi = hi < 0 ? 0 : hi < rows ? hi : rows;
  return {lo, hi > lo ? hi - lo : 0};
}

// s_lo[e], s_n[e]: the experts' rows; s_tile[e]: output tiles of the experts
// before e, at `per` tiles for each `bm` rows begun (s_tile[experts]: all of them).
// By the whole workgroup; ends with a barrier.
__device__ __forceinline__ void expert_tiles(const int* offsets, int experts, int rows, int bm, int per, int* s_lo,
                                             int* s_n, int* s_tile) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int e = e0 + lane;
      ExpertRows r = {0, 0};
      if (e < experts) r = expert_rows(offsets, e, rows);
      const int t = (r.n + bm - 1) / bm * per;
      int x = t;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
      }
      if (e < experts) {
        s_lo[e] = r.lo;
        s_n[e] = r.n;
        s_tile[e] = before + x - t;
      }
      before += __shfl(x, 63);
    }
    if (lane == 0) s_tile[experts] = before;
  }
  __syncthreads();
}

// The expert of tile t, at or after expert e.
__device__ __forceinline__ int expert_of_tile(const int* s_tile, int experts, int t, int e) {
  while (e + 1 < experts && t >= s_tile[e + 1]) ++e;
  return e;
}

}  // namespace pgk
