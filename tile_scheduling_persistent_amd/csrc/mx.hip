// MXFP4 operands: quantisation of a matrix along its rows or (transposed) its
// columns, and the way back.  Each is one pass over the data: a block's
// largest magnitude, its scale byte (integer arithmetic on the magnitude's
// bits) and the conversion, which on gfx950 is one instruction for two values.
// All three are bound by memory: 8192 x 8192 bf16 there and back, 340 MB, in 55
// us (6.2 TB/s); 5000 x 7000 fp32 transposed and back, 247 MB, in 55 us.
//
// Where the tiles fill the device, the wide side goes past the caches,
// non-temporal, if a wave's instructions cover whole lines of it; codes and scales
// stay for the product.  us, plain -> non-temporal, one call on cold data:
//  * values read, 16-bit rows that start on 16 bytes: 8192 x 8192 33.7 -> 29.6,
//    5000 x 7000 22.8 -> 21.6 (4096 x 2056, whose last tile is 8 columns, 9.2 ->
//    10.2); fp32 rows that start on 128-byte lines: 8192 x 8192 60.4 -> 58.0.
//    Other rows have lines that two waves share, which come from memory twice:
//    8192 x 8191 bf16 79.4 -> 83.6, 4096 x 2051 bf16 11.0 -> 12.5, fp32 12.8 -> 14.9.
//  * values written back, 16 bits: 8192 x 8192 36.0 -> 26.2, 8192 x 8191 50.6 ->
//    38.8.  A store of fp32 covers half of each line: 8192 x 8192 80.0 -> 124.5.
// A reader that follows at once finds them in memory instead: both directions of
// 8192 x 8192 bf16 54.4 -> 62.0, values back and a norm of them 80.0 -> 86.3.
#include "common.hpp"
#include "mx_device.hpp"

namespace pgk {
namespace {

constexpr int kThreads = 256;
// Workgroups a launch has at most; past them each takes several tiles (a
// grid's threads have to stay below 2^32).
constexpr int64_t kMaxGrid = 1 << 20;

// Blocks along the columns.  A workgroup takes 4 * RW rows of 512 columns:
// each wave RW whole rows, eight values (16 or 32 bytes) per lane, all RW
// loads in flight before the first is used.  Four lanes share a block of 32
// and exchange its largest magnitude; a row's codes leave as 256 consecutive
// bytes.  The scale bytes of the tile are collected in LDS, because in memory
// the four bytes of a row's 128 columns stand next to those of the next row:
// 32 rows are one 128-byte line.
template <int T, int RW, bool NT>
__global__ void __launch_bounds__(kThreads) quant_kernel(QuantParams p) {
  constexpr int ROWS = 4 * RW;
  __shared__ __attribute__((aligned(4))) unsigned char s_scale[4][ROWS][4];  // read as words
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t groups = (p.cols + 127) / 128, ctiles = (groups + 3) / 4;
  const int64_t tiles = (p.rows + ROWS - 1) / ROWS * ctiles;
  constexpr int esz = T == kTypeF32 ? 4 : 2;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t row0 = rt * ROWS + wave * RW, c = ct * 512 + lane * 8;
    Vec8<T> v[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r < p.rows ? row0 + r : p.rows - 1;
      v[r] = vec8_load<T, false, NT>(static_cast<const char*>(p.X) + row * p.ldx * esz, c, p.cols);
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const unsigned byte = scale_byte<E2M1>(quad_max(vec8_amax(v[r])), p.rule);
      const unsigned o = vec8_e2m1(v[r], scale_value(byte));
      if (row0 + r < p.rows && c < groups * 128)
        *reinterpret_cast<unsigned*>(p.Q + (row0 + r) * groups * 64 + (c >> 1)) = byte == 255u ? 0u : o;
      if ((lane & 3) == 0) s_scale[lane >> 4][wave * RW + r][(lane >> 2) & 3] = (unsigned char)byte;
    }
    __syncthreads();
    if (tid < 4 * ROWS) {
      const int64_t g = ct * 4 + tid / ROWS, row = rt * ROWS + tid % ROWS;
      if (g < groups && row < p.rows)
        reinterpret_cast<unsigned*>(p.scale)[g * p.rows + row] =
            *reinterpret_cast<const unsigned*>(s_scale[tid / ROWS][tid % ROWS]);
    }
    __syncthreads();
  }
}

// Blocks along the rows (the operand of X^T).  A workgroup takes 256 rows of
// 64 columns (fp32; 128 columns of 16 bits, two to a lane): a lane walks down
// its column(s), so a block's 32 values are its own registers and need no
// exchange, and each load of the wave is a row's 256 consecutive bytes.  The
// codes of a column's 256 rows are 128 bytes of one line of the output; they
// pass through LDS so that eight lanes write that line at once.
template <int T>
__global__ void __launch_bounds__(kThreads) quant_transposed_kernel(QuantParams p) {
  constexpr int CPL = T == kTypeF32 ? 1 : 2, COLS = 64 * CPL;
  constexpr int PITCH = 128 + 16;  // bytes of a column's codes in LDS: 16-byte accesses of 16 lanes meet all banks
  __shared__ __attribute__((aligned(16))) unsigned char s_codes[COLS * PITCH];
  __shared__ __attribute__((aligned(4))) unsigned char s_scale[2][COLS][4];  // read as words
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t groups = (p.rows + 127) / 128, rtiles = (groups + 1) / 2, ctiles = (p.cols + COLS - 1) / COLS;
  for (int64_t tile = blockIdx.x; tile < rtiles * ctiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t c = ct * COLS + lane * CPL;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int blk = wave * 2 + h;  // of the tile's eight
      const int64_t k0 = rt * 256 + blk * 32;
      unsigned w[32];
      // rows past the end repeat the last one here and count as zeros below, so
      // that all 32 loads go out together
      const unsigned short* x16 = static_cast<const unsigned short*>(p.X) + c;
      const unsigned* x32 = static_cast<const unsigned*>(p.X) + c;
      if (ct * COLS + COLS <= p.cols) {
        typedef unsigned u32_a2 __attribute__((aligned(2)));
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int64_t at = (k0 + e < p.rows ? k0 + e : p.rows - 1) * p.ldx;
          w[e] = T == kTypeF32 ? x32[at] : *reinterpret_cast<const u32_a2*>(x16 + at);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int64_t at = (k0 + e < p.rows ? k0 + e : p.rows - 1) * p.ldx;
          w[e] = 0u;
          if (c < p.cols) w[e] = T == kTypeF32 ? x32[at] : (unsigned)x16[at];
          if (CPL == 2 && c + 1 < p.cols) w[e] |= (unsigned)x16[at + 1] << 16;
        }
      }
      if (k0 + 32 > p.rows) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (k0 + e >= p.rows) w[e] = 0u;
      }
#pragma unroll
      for (int s = 0; s < CPL; ++s) {
        Vec8<kTypeF32> v[4];
        unsigned amax = 0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float x;
          if (T == kTypeF32)
            x = __builtin_bit_cast(float, w[e]);
          else if (T == kTypeBF16)
            x = __builtin_bit_cast(float, s ? (w[e] & 0xffff0000u) : (w[e] << 16));
          else
            x = (float)__builtin_bit_cast(_Float16, (unsigned short)(s ? (w[e] >> 16) : (w[e] & 0xffffu)));
          const unsigned b = __builtin_bit_cast(unsigned, x);
          v[e >> 3].q[(e >> 2) & 1][e & 3] = b;
          amax = max_u32(amax, b & 0x7fffffffu);
        }
        const unsigned byte = scale_byte<E2M1>(amax, p.rule);
        const float sc = scale_value(byte);
        u32x4_d o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const unsigned code = vec8_e2m1(v[q], sc);
          o[q] = byte == 255u ? 0u : code;
        }
        const int col = lane * CPL + s;
        *reinterpret_cast<u32x4_d*>(s_codes + col * PITCH + blk * 16) = o;
        s_scale[blk >> 2][col][blk & 3] = (unsigned char)byte;
      }
    }
    __syncthreads();
    for (int i = tid; i < COLS * 8; i += kThreads) {
      const int col = i >> 3, q = i & 7;
      const int64_t line = ct * COLS + col, g = rt * 2 + (q >> 2);
      if (line < p.cols && g < groups)
        *reinterpret_cast<Quad<4>::type*>(p.Q + line * groups * 64 + rt * 128 + q * 16) =
            *reinterpret_cast<const u32x4_d*>(s_codes + col * PITCH + q * 16);
    }
    if (tid < 2 * COLS) {
      const int64_t g = rt * 2 + tid / COLS, line = ct * COLS + tid % COLS;
      if (g < groups && line < p.cols)
        reinterpret_cast<unsigned*>(p.scale)[g * p.cols + line] =
            *reinterpret_cast<const unsigned*>(s_scale[tid / COLS][tid % COLS]);
    }
    __syncthreads();
  }
}

// Eight codes per lane, a wave 512 columns of RW rows, their loads in flight
// together.
template <int T, int RW>
__global__ void __launch_bounds__(kThreads) dequant_kernel(DequantParams p) {
  constexpr int ROWS = 4 * RW;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t groups = (p.cols + 127) / 128, ctiles = (p.cols + 511) / 512;
  const int64_t tiles = (p.rows + ROWS - 1) / ROWS * ctiles;
  constexpr int esz = T == kTypeF32 ? 4 : 2;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t rt = tile / ctiles, ct = tile - rt * ctiles;
    const int64_t row0 = rt * ROWS + wave * RW, c = ct * 512 + lane * 8;
    if (c >= p.cols) continue;
    unsigned code[RW], byte[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int64_t row = row0 + r < p.rows ? row0 + r : p.rows - 1;
      code[r] = *reinterpret_cast<const unsigned*>(p.Q + row * groups * 64 + (c >> 1));
      byte[r] = p.scale[((c >> 7) * p.rows + row) * 4 + ((c >> 5) & 3)];
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      if (row0 + r >= p.rows) break;
      float x[8];
      e2m1_values(code[r], byte[r], x);
      vec8_store<T, false, RW == 8 && T != kTypeF32>(static_cast<char*>(p.Y) + (row0 + r) * p.ldy * esz, c, p.cols, vec8_pack<T>(x));
    }
  }
}

dim3 grid_of(int64_t tiles) { return dim3((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid)); }

// Rows per wave: 8 where the tiles still fill the CUs twice over, else 1.
bool tall(int64_t rows, int64_t cols, int cus) { return (rows + 31) / 32 * ((cols + 511) / 512) >= 2 * cus; }

template <int T>
void quant_typed(const QuantParams& p, hipStream_t stream) {
  if (p.transpose) {
    constexpr int COLS = T == kTypeF32 ? 64 : 128;
    const int64_t tiles = (p.rows + 255) / 256 * ((p.cols + COLS - 1) / COLS);
    hipLaunchKernelGGL(quant_transposed_kernel<T>, grid_of(tiles), dim3(kThreads), 0, stream, p);
  } else if (tall(p.rows, p.cols, p.cus)) {
    const dim3 grid = grid_of((p.rows + 31) / 32 * ((p.cols + 511) / 512));
    if (T == kTypeF32 ? rows_at(p.X, p.ldx, 4, 128) : rows_at(p.X, p.ldx, 2, 16))
      hipLaunchKernelGGL((quant_kernel<T, 8, true>), grid, dim3(kThreads), 0, stream, p);
    else
      hipLaunchKernelGGL((quant_kernel<T, 8, false>), grid, dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((quant_kernel<T, 1, false>), grid_of((p.rows + 3) / 4 * ((p.cols + 511) / 512)), dim3(kThreads), 0,
                       stream, p);
  }
}

template <int T>
void dequant_typed(const DequantParams& p, hipStream_t stream) {
  const int64_t ctiles = (p.cols + 511) / 512;
  if (tall(p.rows, p.cols, p.cus))
    hipLaunchKernelGGL((dequant_kernel<T, 8>), grid_of((p.rows + 31) / 32 * ctiles), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((dequant_kernel<T, 1>), grid_of((p.rows + 3) / 4 * ctiles), dim3(kThreads), 0, stream, p);
}

}  // namespace

hipError_t launch_quant(const QuantParams& p, hipStream_t stream) {
  if (p.type == kTypeF32)
    quant_typed<kTypeF32>(p, stream);
  else if (p.type == kTypeBF16)
    quant_typed<kTypeBF16>(p, stream);
  else
    quant_typed<kTypeF16>(p, stream);
  return hipGetLastError();
}

hipError_t launch_dequant(const DequantParams& p, hipStream_t stream) {
  if (p.type == kTypeF32)
    dequant_typed<kTypeF32>(p, stream);
  else if (p.type == kTypeBF16)
    dequant_typed<kTypeBF16>(p, stream);
  else
    dequant_typed<kTypeF16>(p, stream);
  return hipGetLastError();
}

}  // namespace pgk
