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

// Tiles are counted up to here: a program's tile and one stride of the grid more fit in
// an int.  Offsets that rise have fewer; ones that rise and fall, whose ranges share
// rows, may have more, which then no program takes.
constexpr unsigned kMaxTiles = 0x7effffffu;
__device__ __forceinline__ unsigned add_tiles(unsigned a, unsigned b) { return a + b < kMaxTiles ? a + b : kMaxTiles; }

// s_lo[e], s_n[e]: the experts' rows; s_tile[e]: output tiles of the experts
// before e, at `per` tiles for each `bm` rows begun (s_tile[experts]: all of them).
// By the whole workgroup; ends with a barrier.
__device__ __forceinline__ void expert_tiles(const int* offsets, int experts, int rows, int bm, int per, int* s_lo,
                                             int* s_n, int* s_tile) {
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    const ExpertRows r = expert_rows(offsets, e, rows);
    s_lo[e] = r.lo;
    s_n[e] = r.n;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    unsigned before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int e = e0 + lane;
      unsigned x = e < experts ? (unsigned)((s_n[e] + bm - 1) / bm * per) : 0u;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const unsigned y = __shfl_up(x, d);
        if (lane >= d) x = add_tiles(x, y);
      }
      const unsigned up = __shfl_up(x, 1);
      if (e < experts) s_tile[e] = (int)add_tiles(before, lane > 0 ? up : 0u);
      before = add_tiles(before, __shfl(x, 63));
    }
    if (lane == 0) s_tile[experts] = (int)before;
  }
  __syncthreads();
}

// The expert of tile t, at or after expert e: the last one whose tiles start at or
// before t (experts without rows start where the next one does).
__device__ __forceinline__ int expert_of_tile(const int* s_tile, int experts, int t, int e) {
  int end = experts;
  while (end - e > 1) {
    const int mid = (e + end) >> 1;
    if (s_tile[mid] <= t)
      e = mid;
    else
      end = mid;
  }
  return e;
}

}  // namespace pgk
