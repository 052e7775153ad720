// Device helpers of the block-scaled formats: e8m0 scale bytes from block
// magnitudes and the conversions to and from e2m1 / e4m3 (gfx950).
//
// A block's scale exponent is integer arithmetic on the fp32 bits of its
// largest magnitude amax = 1.m * 2^E.  FLOOR: byte = E + 127 - emax.  CEIL
// (smallest e with amax <= top * 2^e, top = 1.t * 2^emax): one more where
// m > t, which is the carry of adding 0x7fffff - t to the bits before the
// shift.  Subnormal and zero magnitudes clamp to byte 0.  Infinities and NaN
// have the largest bits of all magnitudes, so an unsigned maximum carries
// them, and their exponent field 255 is the NaN byte.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pgk {

constexpr int kTypeF32 = 0, kTypeBF16 = 1, kTypeF16 = 2;  // PMX_* element types
constexpr int kRuleCeil = 0, kRuleFloor = 1;              // PMX_SCALE_*

struct E2M1 {
  static constexpr int kEmax = 2;
  static constexpr unsigned kTop = 0x400000u;  // mantissa of 6 = 1.5 * 2^2
};
struct E4M3 {
  static constexpr int kEmax = 8;
  static constexpr unsigned kTop = 0x600000u;  // mantissa of 448 = 1.75 * 2^8
};

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign cleared).
template <class F>
__device__ __forceinline__ unsigned scale_byte(unsigned amax, int rule) {
  if (amax >= 0x7f800000u) return 255u;
  const unsigned up = rule == kRuleCeil ? 0x7fffffu - F::kTop : 0u;
  const int b = (int)((amax + up) >> 23) - F::kEmax;
  return (unsigned)(b < 0 ? 0 : b);
}

// 2^(byte - 127) as fp32; byte 255 gives NaN.
__device__ __forceinline__ float scale_value(unsigned byte) {
  const unsigned bits = byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
  return __builtin_bit_cast(float, bits);
}

typedef __bf16 bf16x2_d __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_d __attribute__((ext_vector_type(2)));
typedef float f32x2_d __attribute__((ext_vector_type(2)));
typedef short s16x2_d __attribute__((ext_vector_type(2)));
typedef unsigned u32x2_d __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_d __attribute__((ext_vector_type(4)));

// Eight consecutive elements as stored: 16 bytes (16-bit types) or 32 (fp32).
template <int T>
struct Vec8 {
  u32x4_d q[T == kTypeF32 ? 2 : 1];
};

// Element e of the eight as fp32.
template <int T>
__device__ __forceinline__ float vec8_get(const Vec8<T>& v, int e) {
  // the element first, then the cast: a bit cast of a vector element itself
  // reads element 0
  const unsigned w = T == kTypeF32 ? v.q[e >> 2][e & 3] : v.q[0][e >> 1];
  if (T == kTypeF32) return __builtin_bit_cast(float, w);
  if (T == kTypeBF16) return __builtin_bit_cast(float, (e & 1) ? (w & 0xffff0000u) : (w << 16));
  return (float)__builtin_bit_cast(_Float16, (unsigned short)((e & 1) ? (w >> 16) : (w & 0xffffu)));
}

// Eight fp32 values rounded (to nearest even) to the stored form.
template <int T>
__device__ __forceinline__ Vec8<T> vec8_pack(const float (&x)[8]) {
  Vec8<T> v;
  if (T == kTypeF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v.q[e >> 2][e & 3] = __builtin_bit_cast(unsigned, x[e]);
  } else if (T == kTypeBF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v.q[0][e] = __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2_d{x[2 * e], x[2 * e + 1]}, bf16x2_d));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v.q[0][e] = __builtin_bit_cast(unsigned, f16x2_d{(_Float16)x[2 * e], (_Float16)x[2 * e + 1]});
  }
  return v;
}

// 16 bytes at an address aligned to `A` bytes: global memory accesses of any
// alignment are single instructions here, so rows that start on odd elements
// move as wide as aligned ones.
template <int A>
struct Quad;
template <>
struct Quad<4> {
  typedef u32x4_d __attribute__((aligned(4))) type;
};
template <>
struct Quad<2> {
  typedef u32x4_d __attribute__((aligned(2))) type;
};

// Elements i .. i + 7 of a row that ends at `n` (elements past it zero).
// WHOLE: n is a multiple of 8, as i is, and the code for a vector's part falls
// away.
template <int T, bool WHOLE = false, bool NT = false>
__device__ __forceinline__ Vec8<T> vec8_load(const void* row, int64_t i, int64_t n) {
  constexpr int esz = T == kTypeF32 ? 4 : 2;
  Vec8<T> v;
#pragma unroll
  for (int q = 0; q < esz / 2; ++q) v.q[q] = u32x4_d{0, 0, 0, 0};
  if (i + 8 <= n) {
    const auto* p = reinterpret_cast<const typename Quad<esz>::type*>(static_cast<const char*>(row) + i * esz);
#pragma unroll
    for (int q = 0; q < esz / 2; ++q) {
      if constexpr (NT)
        v.q[q] = __builtin_nontemporal_load(p + q);
      else
        v.q[q] = p[q];
    }
  } else if (!WHOLE && i < n) {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (i + e >= n) continue;
      if (T == kTypeF32)
        v.q[e >> 2][e & 3] = static_cast<const unsigned*>(row)[i + e];
      else
        v.q[0][e >> 1] |= (unsigned)static_cast<const unsigned short*>(row)[i + e] << (16 * (e & 1));
    }
  }
  return v;
}

template <int T, bool WHOLE = false, bool NT = false>
__device__ __forceinline__ void vec8_store(void* row, int64_t i, int64_t n, const Vec8<T>& v) {
  constexpr int esz = T == kTypeF32 ? 4 : 2;
  if (i + 8 <= n) {
    auto* p = reinterpret_cast<typename Quad<esz>::type*>(static_cast<char*>(row) + i * esz);
#pragma unroll
    for (int q = 0; q < esz / 2; ++q) {
      if constexpr (NT)
        __builtin_nontemporal_store(v.q[q], p + q);
      else
        p[q] = v.q[q];
    }
  } else if (!WHOLE && i < n) {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (i + e >= n) continue;
      if (T == kTypeF32)
        static_cast<unsigned*>(row)[i + e] = v.q[e >> 2][e & 3];
      else
        static_cast<unsigned short*>(row)[i + e] = (unsigned short)(v.q[0][e >> 1] >> (16 * (e & 1)));
    }
  }
}

// Every row of a matrix starts at a multiple of `align` (a power of two) bytes.
inline bool rows_at(const void* x, int64_t ld, int64_t esz, int64_t align) {
  return (reinterpret_cast<uintptr_t>(x) & (uintptr_t)(align - 1)) == 0 && (ld * esz & (align - 1)) == 0;
}

// Largest over the 4 lanes of a quad, and over the 16 lanes of a row, in
// every lane of it (data-parallel primitives: no LDS).
__device__ __forceinline__ unsigned max_u32(unsigned a, unsigned b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned quad_max(unsigned m) {
  m = max_u32(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));     // lanes 1 0 3 2
  return max_u32(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // lanes 2 3 0 1
}
__device__ __forceinline__ unsigned row16_max(unsigned m) {
  m = quad_max(m);
  m = max_u32(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));    // rotated by 4
  return max_u32(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, true)); // rotated by 8
}

// Largest magnitude of the eight, as fp32 bits.
template <int T>
__device__ __forceinline__ unsigned vec8_amax(const Vec8<T>& v) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned b = __builtin_bit_cast(unsigned, vec8_get(v, e)) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}

// The eight as e2m1 codes in units of `scale` (a power of two), the first in
// the low nibble: rounded to nearest even, saturating at 6.
template <int T>
__device__ __forceinline__ unsigned vec8_e2m1(const Vec8<T>& v, float scale) {
  unsigned o = 0;
  if (T == kTypeBF16) {
    const unsigned w0 = v.q[0][0], w1 = v.q[0][1], w2 = v.q[0][2], w3 = v.q[0][3];
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_d, w0), scale, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_d, w1), scale, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_d, w2), scale, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2_d, w3), scale, 3);
  } else {
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, vec8_get(v, 0), vec8_get(v, 1), scale, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, vec8_get(v, 2), vec8_get(v, 3), scale, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, vec8_get(v, 4), vec8_get(v, 5), scale, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, vec8_get(v, 6), vec8_get(v, 7), scale, 3);
  }
  return o;
}

// The values of eight e2m1 codes under scale byte `byte`, fp32 (exact; past
// the range infinity).  ldexp rather than a product: a product that is rounded
// to fp16 next becomes a fused multiply-add of zero, which loses the sign of
// negative zeros.
__device__ __forceinline__ void e2m1_values(unsigned codes, unsigned byte, float (&x)[8]) {
  const f32x2_d a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const f32x2_d b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const f32x2_d c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const f32x2_d d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    x[e] = byte == 255u ? __builtin_nanf("") : __builtin_ldexpf(v[e], (int)byte - 127);
}

}  // namespace pgk
