// Tokens routed to experts: the slots (token, choice) sorted by expert, the
// tokens' rows in that order, the experts' rows back at their tokens, and the
// gradients of that.
//
// The sort is a stable counting sort, so its result does not depend on the order
// in which waves run.  Everything else works row by row, and is bound by memory.
// Indices that come from device memory are checked against the sizes of the call
// before they are used: a wrong one leaves its row out.
#include "common.hpp"
#include "fp8_rows.hpp"

namespace pgk {
namespace {

// ------------------------------------------------------------------- the sort
//
// A slot's row is its expert's first row, plus the slots of that expert in earlier
// parts of the slots (a part to a workgroup) and in earlier waves of the part, plus
// the equal lanes below it in its wave.

template <typename I>
__device__ __forceinline__ int expert_in(const SortParams& p, I id) {
  return id >= 0 && id < p.experts ? (int)id : -1;
}

// Lanes with the same expert as this one (experts below 2^bits).
__device__ __forceinline__ unsigned long long same_lanes(int e, int bits) {
  unsigned long long m = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool on = (e >> b) & 1;
    const unsigned long long v = __ballot(on);
    m &= on ? v : ~v;
  }
  return m;
}

// Adds a slot to counts in LDS, kCopies of each: atomics on one word take turns, and
// routers have favourites.
constexpr int kCopies = 4;
__device__ __forceinline__ void count_slot(int e, int* cnt) {
  if (e >= 0) atomicAdd(cnt + e * kCopies + (threadIdx.x & (kCopies - 1)), 1);
}
__device__ __forceinline__ int counted(const int* cnt, int e) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < kCopies; ++i) n += cnt[e * kCopies + i];
  return n;
}

// Exclusive prefix sums over the workgroup's threads; *total: the sum.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int* s_wave, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) s_wave[wave] = x;
  __syncthreads();
  int base = 0, all = 0;
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) base += s_wave[w];
    all += s_wave[w];
  }
  *total = all;
  __syncthreads();
  return base + x - v;
}

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
static_assert(kMaxExperts <= kSortThreads, "a thread per expert");

// Rows of the slots of one part, a slot per thread, from each expert's first row of
// the part (`at`, thread e's), by way of s_cnt [waves][experts].
template <typename I>
__device__ __forceinline__ void place_part(const SortParams& p, int64_t begin, int64_t end, int at, int* s_cnt, bool order) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
  for (int64_t s0 = begin; s0 < end; s0 += kSortThreads) {
    for (int i = tid; i < kSortWaves * E; i += kSortThreads) s_cnt[i] = 0;
    __syncthreads();
    const int64_t s = s0 + tid;
    const int e = s < end ? expert_in(p, static_cast<const I*>(p.ids)[s]) : -1;
    const unsigned long long m = same_lanes(e, p.bits);
    const int below = __popcll(m & ((1ull << lane) - 1ull));
    if (e >= 0 && below == 0) s_cnt[wave * E + e] = __popcll(m);
    __syncthreads();
    if (tid < E)
      for (int w = 0; w < kSortWaves; ++w) {
        const int n = s_cnt[w * E + tid];
        s_cnt[w * E + tid] = at;
        at += n;
      }
    __syncthreads();
    if (s < end) {
      const int row = e >= 0 ? s_cnt[wave * E + e] + below : -1;
      p.place[s] = row;
      if (order && e >= 0) p.order[row] = (int)s;
    }
    __syncthreads();
  }
}

// One launch: every workgroup counts all slots, those before its part and the
// others, in LDS.  Counting again what the others count costs less than launches that
// pass counts on up to some ten thousand slots (64 experts, us: 32768 slots 8.8; 65536
// slots 13.3, and 12.0 in three launches).
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortParams p) {
  extern __shared__ int s_cnt[];  // [waves][experts]; before that [2][experts][copies]
  __shared__ int s_wave[kSortWaves];
  const int tid = threadIdx.x, E = p.experts;
  int* s_before = s_cnt;
  int* s_rest = s_cnt + E * kCopies;
  for (int i = tid; i < 2 * E * kCopies; i += kSortThreads) s_cnt[i] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * kSortThreads;
  const int64_t end = begin + kSortThreads < p.slots ? begin + kSortThreads : p.slots;
  constexpr int AT_ONCE = 4;  // loads on their way together
  for (int64_t s0 = 0; s0 < p.slots; s0 += AT_ONCE * kSortThreads) {
    I id[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int64_t s = s0 + i * kSortThreads + tid;
      id[i] = s < p.slots ? static_cast<const I*>(p.ids)[s] : (I)-1;
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) count_slot(expert_in(p, id[i]), s0 + i * kSortThreads < begin ? s_before : s_rest);
  }
  __syncthreads();
  const int before = tid < E ? counted(s_before, tid) : 0, all = tid < E ? before + counted(s_rest, tid) : 0;
  int total;
  const int at = block_prefix<kSortThreads>(all, s_wave, &total);
  if (blockIdx.x == 0) {
    if (tid < E) p.offsets[tid] = at;
    if (tid == 0) p.offsets[E] = total;
  }
  place_part<I>(p, begin, end, at + before, s_cnt, true);
  if (begin + tid < end && begin + tid >= total) p.order[begin + tid] = -1;
}

// More slots: a count per workgroup and expert, kept in `order` until the last of
// three launches writes that.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortParams p) {
  extern __shared__ int s_cnt[];  // [experts][copies]
  const int E = p.experts;
  for (int i = threadIdx.x; i < E * kCopies; i += kSortThreads) s_cnt[i] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * p.part, end = begin + p.part < p.slots ? begin + p.part : p.slots;
  for (int64_t s0 = begin; s0 < end; s0 += kSortThreads) {
    const int64_t s = s0 + threadIdx.x;
    count_slot(s < end ? expert_in(p, static_cast<const I*>(p.ids)[s]) : -1, s_cnt);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kSortThreads) p.order[(int64_t)blockIdx.x * E + i] = counted(s_cnt, i);
}

template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p) {
  extern __shared__ int s_cnt[];  // [waves][experts]; before that [2][experts]
  __shared__ int s_wave[kSortWaves];
  const int tid = threadIdx.x, E = p.experts;
  int* s_before = s_cnt;
  int* s_all = s_cnt + E;
  if (tid < E) s_before[tid] = s_all[tid] = 0;
  __syncthreads();
  const int lanes = kSortThreads / E;  // threads per expert
  if (tid < lanes * E) {
    const int e = tid % E;
    int all = 0, before = 0;
    for (int b = tid / E; b < p.parts; b += lanes) {
      const int n = p.order[(int64_t)b * E + e];
      all += n;
      before += b < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(s_all + e, all);
    atomicAdd(s_before + e, before);
  }
  __syncthreads();
  const int all = tid < E ? s_all[tid] : 0, before = tid < E ? s_before[tid] : 0;
  int total;
  const int at = block_prefix<kSortThreads>(all, s_wave, &total);
  if (blockIdx.x == 0) {
    if (tid < E) p.offsets[tid] = at;
    if (tid == 0) p.offsets[E] = total;
  }
  const int64_t begin = blockIdx.x * p.part, end = begin + p.part < p.slots ? begin + p.part : p.slots;
  place_part<I>(p, begin, end, at + before, s_cnt, false);
}

__global__ void __launch_bounds__(256) sort_order_kernel(SortParams p) {
  const int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (s >= p.slots) return;
  const int total = p.offsets[p.experts], row = p.place[s];
  if (row >= 0) p.order[row] = (int)s;
  if (s >= total) p.order[s] = -1;
}

template <typename I>
hipError_t sort_typed(SortParams p, hipStream_t stream) {
  const int lds = kSortWaves * p.experts * (int)sizeof(int);
  static_assert(kSortWaves >= 2 * kCopies, "the first counts fit where the waves' counts go");
  auto allow = [&](const void* kern) {
    if (lds > 65536 - 256) (void)hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  };
  if (p.slots <= kSortOnce) {
    allow((const void*)sort_kernel<I>);
    const unsigned grid = p.slots > 0 ? (unsigned)((p.slots + kSortThreads - 1) / kSortThreads) : 1u;
    hipLaunchKernelGGL(sort_kernel<I>, dim3(grid), dim3(kSortThreads), lds, stream, p);
    return hipGetLastError();
  }
  // at most 256 parts, of at least two slots per expert: their counts fit in `order`
  p.part = (p.slots + 255) / 256 > 2 * p.experts ? (p.slots + 255) / 256 : 2 * p.experts;
  p.part = (p.part + kSortThreads - 1) / kSortThreads * kSortThreads;
  static_assert(kSortOnce >= 2 * kMaxExperts, "and those of the last one");
  p.parts = (int)((p.slots + p.part - 1) / p.part);
  allow((const void*)sort_place_kernel<I>);
  hipLaunchKernelGGL(sort_count_kernel<I>, dim3(p.parts), dim3(kSortThreads), p.experts * kCopies * sizeof(int), stream, p);
  hipLaunchKernelGGL(sort_place_kernel<I>, dim3(p.parts), dim3(kSortThreads), lds, stream, p);
  hipLaunchKernelGGL(sort_order_kernel, dim3((unsigned)((p.slots + 255) / 256)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

// ------------------------------------------------------- rows by sorted slots

// The slot of a row, -1 where it has none.
__device__ __forceinline__ int slot_of(const int* order, int64_t row, int64_t slots) {
  const int s = row < slots ? order[row] : -1;
  return s >= 0 && s < slots ? s : -1;
}

// A workgroup takes 128 columns of 16 * R rows, 16 lanes to a row.  The tiles of eight
// stretches of 128 columns go round the XCDs, all rows before the next eight: an
// XCD's workgroups then read the same 256 bytes of every token (16 bits), 2 MiB of
// 8192 tokens, which stay in its L2 although a token is read for each of its slots in
// the order of the experts (8192 x 8 x 4096 to e4m3, with the sort: a row's columns side
// by side 105.6 us, so 83).  NT: the output goes past the caches, where the tokens stay for
// their other slots (gather_typed has the rule).
template <int T, int R, bool QUANT, bool NT>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(GatherParams p) {
  constexpr int ROWS = 16 * R;
  __shared__ unsigned char s_scale[ROWS];
  __shared__ int s_slot[ROWS];
  const int tid = threadIdx.x, lane16 = tid & 15, sub = tid >> 4;
  const int64_t slots = p.tokens * p.topk, groups = (p.cols + 127) / 128, kp = groups * 128;
  const int64_t rtiles = (slots + ROWS - 1) / ROWS, tiles = rtiles * groups;
  const double per_topk = 1.0 / (double)p.topk;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t eight = tile / (8 * rtiles), in = tile - eight * 8 * rtiles;
    const int64_t wide = groups - eight * 8 < 8 ? groups - eight * 8 : 8;
    const int64_t rt = in / wide, g = eight * 8 + in - rt * wide;
    const int64_t c = g * 128 + lane16 * 8;
    int slot[R];
    Vec8<T> v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) slot[r] = slot_of(p.order, rt * ROWS + r * 16 + sub, slots);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // slot / topk: a 64-bit product is off by less than the half
      const int token = slot[r] >= 0 ? (int)(((double)slot[r] + 0.5) * per_topk) : 0;
      v[r] = vec8_load<T>(static_cast<const char*>(p.X) + token * p.ldx * size_of(T), c, p.cols);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = rt * ROWS + r * 16 + sub;
      if (QUANT) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = vec8_get(v[r], e);
        unsigned byte;
        const u32x2_d o = e4m3_codes(x, byte);
        if (slot[r] >= 0) {
          u32x2_d* q = reinterpret_cast<u32x2_d*>(static_cast<uint8_t*>(p.Y) + row * kp + c);
          if constexpr (NT)
            __builtin_nontemporal_store(o, q);
          else
            *q = o;
        }
        if (lane16 == 0) {
          s_scale[r * 16 + sub] = (unsigned char)byte;
          s_slot[r * 16 + sub] = slot[r];
        }
      } else if (slot[r] >= 0) {
        vec8_store<T, false, NT>(static_cast<char*>(p.Y) + row * p.ldy * size_of(T), c, p.cols, v[r]);
      }
    }
    if (QUANT) {
      __syncthreads();
      if (tid < ROWS && s_slot[tid] >= 0) p.y_scale[g * slots + rt * ROWS + tid] = s_scale[tid];
      __syncthreads();
    }
  }
}

// A wave takes 512 columns of a token: up to eight of its slots' rows at a time
// are on their way together, summed in fp32 in the slots' order.
// NT: rows and result past the caches, where the rows fill most of the Infinity Cache, in
// every type and wherever rows start (a row is read once, and most of what moves is read).
// us, past them / through them, with a norm of the result: 8192 x 8 x 4096 bf16 139 / 162,
// alone 108 / 130; 2048 tokens 40.2 / 43.2; 1024 tokens, whose rows may still be there, 25.0
// / 22.2.  bf16 8192 x 8, a stride of 4104 121 / 131, 5000 columns 158 / 162, 4095 columns 204
// / 207, to fp32 137 / 151; fp32 4096 x 8 x 4096 122 / 131, 4095 columns 146 / 152, 1100 x 8 x
// 4096 38.3 / 38.5.
constexpr int kSlotsAtOnce = 8;
template <int T, int YT, bool NT>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(CombineParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t slots = p.tokens * p.topk, ctiles = (p.cols + kRowCols - 1) / kRowCols;
  const int64_t tiles = p.tokens * ctiles;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t tile = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); tile < tiles; tile += step) {
    const int64_t t = tile / ctiles, c = (tile - t * ctiles) * kRowCols + lane * 8;
    float y[8] = {};
    Vec8<YT> res;
    if (p.R) res = vec8_load<YT>(static_cast<const char*>(p.R) + t * p.ldr * size_of(YT), c, p.cols);
    for (int j0 = 0; j0 < p.topk; j0 += kSlotsAtOnce) {
      Vec8<T> v[kSlotsAtOnce];
      float w[kSlotsAtOnce];
#pragma unroll
      for (int j = 0; j < kSlotsAtOnce; ++j) {
        const int64_t s = t * p.topk + j0 + j;
        const int row = j0 + j < p.topk ? p.place[s] : -1;
        const bool on = row >= 0 && row < slots;
        w[j] = on ? (p.weights ? p.weights[s] : 1.0f) : 0.0f;
        v[j] = vec8_load<T, false, NT>(static_cast<const char*>(p.X) + (on ? row : 0) * p.ldx * size_of(T), c, on ? p.cols : 0);
      }
#pragma unroll
      for (int j = 0; j < kSlotsAtOnce; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(w[j], vec8_get(v[j], e), y[e]);
    }
    if (p.R) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += vec8_get(res, e);
    }
    vec8_store<YT, false, NT>(static_cast<char*>(p.Y) + t * p.ldy * size_of(YT), c, p.cols, vec8_pack<YT>(y));
  }
}

// A wave takes RW rows, all of their columns: dx = w dy, and the dot product of
// dy with the row for dw.  NT: rows in and out past the caches, which leaves those to dy
// that is read for each slot (combine_grad_typed has the rule).
template <int T, int RW, bool QUANT, bool NT>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(CombineGradParams p) {
  constexpr int ROWS = 4 * RW;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t slots = p.tokens * p.topk, kp = (p.cols + 127) / 128 * 128;
  const int64_t tiles = (slots + ROWS - 1) / ROWS;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t row0 = tile * ROWS + wave * RW;
    int slot[RW];
    float w[RW], dot[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      slot[r] = slot_of(p.order, row0 + r, slots);
      w[r] = slot[r] >= 0 && p.weights ? p.weights[slot[r]] : 1.0f;
      dot[r] = 0.0f;
    }
    for (int64_t c = lane * 8; c - lane * 8 < p.cols; c += kRowCols) {
      Vec8<T> d[RW], x[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const int64_t token = slot[r] >= 0 ? (unsigned)slot[r] / (unsigned)p.topk : 0;
        const int64_t n = slot[r] >= 0 ? p.cols : 0;
        d[r] = vec8_load<T>(static_cast<const char*>(p.dY) + token * p.ldy * size_of(T), c, n);
        if (p.dW) x[r] = vec8_load<T, false, NT>(static_cast<const char*>(p.X) + (slot[r] >= 0 ? row0 + r : 0) * p.ldx * size_of(T), c, n);
      }
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = vec8_get(d[r], e);
          if (p.dW) dot[r] = __builtin_fmaf(y[e], vec8_get(x[r], e), dot[r]);
          y[e] *= w[r];
        }
        if (QUANT) {
          if (c + 8 > p.cols) {  // the padding is zero whatever the weight is
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c + e >= p.cols) y[e] = 0.0f;
          }
          unsigned byte;
          const u32x2_d o = e4m3_codes(y, byte);
          if (slot[r] >= 0 && c < kp) {
            u32x2_d* q = reinterpret_cast<u32x2_d*>(static_cast<uint8_t*>(p.dX) + (row0 + r) * kp + c);
            if constexpr (NT)
              __builtin_nontemporal_store(o, q);
            else
              *q = o;
            if ((lane & 15) == 0) p.dx_scale[(c >> 7) * slots + row0 + r] = (uint8_t)byte;
          }
        } else if (slot[r] >= 0) {
          vec8_store<T, false, NT>(static_cast<char*>(p.dX) + (row0 + r) * p.lddx * size_of(T), c, p.cols, vec8_pack<T>(y));
        }
      }
    }
    if (p.dW) {
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float v = dot[r];
#pragma unroll
        for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
        if (lane == 0 && slot[r] >= 0) p.dW[slot[r]] = v;
      }
      // slots that no row has
      for (int i = threadIdx.x; i < ROWS; i += kRowThreads) {
        const int64_t s = tile * ROWS + i;
        if (s < slots && (p.place[s] < 0 || p.place[s] >= slots)) p.dW[s] = 0.0f;
      }
    }
  }
}

constexpr int64_t kPastCaches = 128ll << 20;

// Past the caches go codes of any size, which 16 lanes write by whole lines, and rows of 16
// bits that would fill most of the Infinity Cache, where they start on lines.  us, past them
// / through them.  Codes, with the product that reads them next: 16 MB 61 / 72, 256 MB 404
// / 448; alone 8.0 / 12.3 and 76 / 167.  bf16, 8192 x 8 x 4096: 128 / 173; rows that start
// on 16 bytes (a stride of 4104) 250 / 248, of 5000 columns 321 / 289, of 4095 305 / 280.  An
// access of fp32 covers half of each line: 4096 x 8 x 4096 259 / 163, 4095 columns 317 / 239.
template <int T, bool QUANT>
void gather_typed(const GatherParams& p, hipStream_t stream) {
  const int64_t slots = p.tokens * p.topk, groups = (p.cols + 127) / 128, tall = (slots + 127) / 128 * groups;
  const dim3 block(kRowThreads);
  if (tall < 4 * p.cus) {
    hipLaunchKernelGGL((gather_kernel<T, 1, QUANT, false>), row_grid((slots + 15) / 16 * groups), block, 0, stream, p);
    return;
  }
  if constexpr (QUANT || T != kTypeF32) {
    if (QUANT || (slots * p.cols * size_of(T) >= kPastCaches && rows_at(p.Y, p.ldy, size_of(T), 128))) {
      hipLaunchKernelGGL((gather_kernel<T, 8, QUANT, true>), row_grid(tall), block, 0, stream, p);
      return;
    }
  }
  if constexpr (!QUANT) hipLaunchKernelGGL((gather_kernel<T, 8, false, false>), row_grid(tall), block, 0, stream, p);
}
template <int T>
void gather_out(const GatherParams& p, hipStream_t stream) {
  p.y_scale ? gather_typed<T, true>(p, stream) : gather_typed<T, false>(p, stream);
}

template <int T, int YT>
void combine_typed(const CombineParams& p, hipStream_t stream) {
  const dim3 grid = row_grid((p.tokens * ((p.cols + kRowCols - 1) / kRowCols) + 3) / 4), block(kRowThreads);
  if (p.tokens * p.topk * p.cols * size_of(T) >= kPastCaches)
    hipLaunchKernelGGL((combine_kernel<T, YT, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((combine_kernel<T, YT, false>), grid, block, 0, stream, p);
}
template <int T>
void combine_out(const CombineParams& p, hipStream_t stream) {
  p.y_type == T ? combine_typed<T, T>(p, stream) : combine_typed<T, kTypeF32>(p, stream);
}

// Rows that fill most of the Infinity Cache go past the caches, but for fp32 results that
// start on lines, of which an access covers half of each.  us, past them / through them:
// 8192 x 8 x 4096 bf16 241 / 250, without dw 159 / 169, to e4m3 207 / 214; 4095 columns 286 /
// 314, 168 / 226 and 265 / 270; rows that fit, 512 x 8 x 4096, 17.0 / 15.3.  fp32, 4096 x 8 x
// 4096 294 / 274 and 210 / 173, to e4m3 192 / 199; rows off lines, 4095 columns 297 / 295 and
// 204 / 230, a stride of 4100 293 / 294 and 207 / 226.
template <int T, bool QUANT>
void combine_grad_typed(const CombineGradParams& p, hipStream_t stream) {
  const int64_t slots = p.tokens * p.topk;
  const dim3 block(kRowThreads);
  const bool half_lines = T == kTypeF32 && !QUANT && rows_at(p.dX, p.lddx, size_of(T), 128);
  if ((slots + 15) / 16 < 2 * p.cus)
    hipLaunchKernelGGL((combine_grad_kernel<T, 1, QUANT, false>), row_grid((slots + 3) / 4), block, 0, stream, p);
  else if (slots * p.cols * size_of(T) < kPastCaches || half_lines)
    hipLaunchKernelGGL((combine_grad_kernel<T, 4, QUANT, false>), row_grid((slots + 15) / 16), block, 0, stream, p);
  else
    hipLaunchKernelGGL((combine_grad_kernel<T, 4, QUANT, true>), row_grid((slots + 15) / 16), block, 0, stream, p);
}
template <int T>
void combine_grad_out(const CombineGradParams& p, hipStream_t stream) {
  p.dx_scale ? combine_grad_typed<T, true>(p, stream) : combine_grad_typed<T, false>(p, stream);
}

}  // namespace

hipError_t launch_sort(const SortParams& p, hipStream_t stream) {
  return p.ids64 ? sort_typed<int64_t>(p, stream) : sort_typed<int32_t>(p, stream);
}

#define PGK_BY_TYPE(type, fn)       \
  do {                              \
    if ((type) == kTypeF32)         \
      fn<kTypeF32>(p, stream);      \
    else if ((type) == kTypeBF16)   \
      fn<kTypeBF16>(p, stream);     \
    else                            \
      fn<kTypeF16>(p, stream);      \
    return hipGetLastError();       \
  } while (0)

hipError_t launch_gather(const GatherParams& p, hipStream_t stream) { PGK_BY_TYPE(p.type, gather_out); }
hipError_t launch_combine(const CombineParams& p, hipStream_t stream) { PGK_BY_TYPE(p.type, combine_out); }
hipError_t launch_combine_grad(const CombineGradParams& p, hipStream_t stream) { PGK_BY_TYPE(p.type, combine_grad_out); }

}  // namespace pgk
