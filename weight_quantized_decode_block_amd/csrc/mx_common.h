// The microscaled formats on gfx950: conversions shared by the quantisation,
// norm and product kernels.
//
// A block of 32 values along a row shares an E8M0 scale byte s that stands
// for 2^(s - 127) (255: NaN).  MXFP4 elements are E2M1 (0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives), two a byte with the even element in the low
// nibble; MXFP8 elements are E4M3FN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace wqd {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// f(integral_constant<D>) for D = B .. E-1, unrolled at compile time
template <int B, int E, typename F>
__device__ __forceinline__ void mx_unroll(F &&f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    mx_unroll<B + 1, E>(f);
  }
}

// Two fp32 as BF16, round to nearest even, `a` in the low half
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The value of an E8M0 byte: 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  const uint32_t bits = s == 0u ? 0x00400000u : s << 23;
  return __uint_as_float(s == 255u ? 0x7fc00000u : bits);
}

constexpr uint32_t kFp4Emax = 2;  // 6 = 1.5 * 2^2 is the largest E2M1 value
constexpr uint32_t kFp8Emax = 8;  // 448 = 1.75 * 2^8 is the largest E4M3FN value

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (integer order: infinities and NaN come out on top): floor(log2 amax) - emax
// + 127 from the exponent field, not below 0 (a subnormal or zero amax has
// field 0), 255 for a block with a value that is not finite.
template <uint32_t EMAX>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t f = amax >> 23;
  return f == 255u ? 255u : (f > EMAX ? f - EMAX : 0u);
}

// 2^(127 - s): what the block's values are multiplied by before they are
// rounded (always a normal number, so the product is exact unless it is far
// below the smallest element).  0 for s = 255, whose codes are all 0.
__device__ __forceinline__ float mx_inverse(uint32_t s) {
  return __uint_as_float(s == 255u ? 0u : (254u - s) << 23);
}

// max over a block's four lanes (lanes 4i .. 4i+3 of a wave hold 8 values each)
__device__ __forceinline__ uint32_t max_of_4_lanes(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false);  // neighbour
  x = x > y ? x : y;
  const uint32_t z = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false);  // other pair
  return x > z ? x : z;
}

// 8 scaled values as E2M1 codes (the hardware conversion: round to nearest
// even, saturated at 6, the sign of a zero kept)
__device__ __forceinline__ uint32_t fp4x8(const float (&v)[8]) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
  return r;
}

// 8 scaled values as E4M3FN bytes, clamped first: the conversion turns what
// rounds above 448 into NaN
__device__ __forceinline__ u32x2_t fp8x8(const float (&v)[8]) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -448.0f, 448.0f);
  u32x2_t r;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  return r;
}

}  // namespace wqd
