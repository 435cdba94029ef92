// mxfp4_device.h -- device-side helpers of the MXFP4 kernels: the block rule on
// a few lanes, and the types of the scaled matrix instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4_launch.h"
#include "q8_device.h"

namespace mx {

using q8::f32x16;
using q8::f32x4;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;

// Eight consecutive unquantized values of a lane, in the bits they have in memory.
template <int TYPE>
struct Eight {
  uint32_t d[TYPE == kF32 ? 8 : 4];
};

// Bits of max|v_i| as an fp32 number; 0x7F800000 and above if a value is not finite.
template <int TYPE>
__device__ __forceinline__ uint32_t amax_bits(const Eight<TYPE> &v) {
  uint32_t m = 0;
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v.d[i] & 0x7FFFFFFFu);
  } else if constexpr (TYPE == kBF16) {  // a bf16 number is the high half of an fp32 one
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((v.d[i] << 16) & 0x7FFFFFFFu, v.d[i] & 0x7FFF0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(v.d[i] & 0x7FFFu, (v.d[i] >> 16) & 0x7FFFu));
    m = __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m));
  }
  return m;
}

// The maximum over aligned groups of four lanes, in each of them.
__device__ __forceinline__ uint32_t max_quad(uint32_t m) {
  m = max(m, q8::dpp_u32<q8::kDppXor1>(m));
  return max(m, q8::dpp_u32<q8::kDppXor2>(m));
}

// The scale byte of a block with this amax.  floor(log2 amax) of a normal
// number is its exponent field - 127; below 2^-124 the scale is 2^-127.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e >= 255 ? 255u : (e > 2 ? e - 2 : 0u);
}

// 2^(byte - 127) in fp32 (byte 0 is the subnormal 2^-127; 255 gives infinity).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// Eight codes, value i in bits 4i..4i+3.  The convert divides by the scale,
// rounds to nearest even and saturates at 6 (checked over every binade of the
// three types, subnormal inputs and scales included).
template <int TYPE>
__device__ __forceinline__ uint32_t encode(const Eight<TYPE> &v, uint32_t byte) {
  if (byte == 255) return 0;
  const float s = scale_value(byte);
  uint32_t r = 0;
  if constexpr (TYPE == kF32) {
    auto f = [&](int i) { return __builtin_bit_cast(float, v.d[i]); };
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(0), f(1), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(2), f(3), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(4), f(5), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f(6), f(7), s, 3);
  } else if constexpr (TYPE == kBF16) {
    auto f = [&](int i) { return __builtin_bit_cast(bf16x2, v.d[i]); };
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, f(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, f(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, f(2), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, f(3), s, 3);
  } else {
    auto f = [&](int i) { return __builtin_bit_cast(f16x2, v.d[i]); };
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, f(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, f(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, f(2), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, f(3), s, 3);
  }
  return r;
}

// fp32 to bf16 / fp16 bits, to nearest even (overflow to infinity, NaN kept).
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t f16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}

}  // namespace mx
