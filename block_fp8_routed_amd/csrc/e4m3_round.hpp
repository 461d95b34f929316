// e4m3_round.hpp — the E4M3 rounding and block-exponent rule of the FP8
// variant (activations and the SwiGLU output h), shared by the activation
// quantiser and the FP8 gate/up pass.
//
// Reading of this project (the pages describe E4M3 weights only): a block of
// 128 values gets the scale 2^e, e the smallest integer with max|v| <= 448 *
// 2^e (0 for an all-zero block, at least -127); each value becomes the
// nearest OCP E4M3FN value of v * 2^-e, ties to the even mantissa, sign kept.
#pragma once

#include "device.hpp"

namespace moe {

constexpr int kActBlock = 128;  // columns per activation scale block

// nearest E4M3FN byte to v, |v| <= 448 (ties to the even mantissa, sign kept)
__device__ __forceinline__ uint32_t e4m3_rne(float v) {
  const uint32_t sign = (__float_as_uint(v) >> 31) << 7;
  const float a = fabsf(v);
  uint32_t code;
  if (a < 0x1p-6f) {
    // subnormal range: m * 2^-9 with m = 0 .. 8 (m = 8 is the smallest
    // normal, code 0x08)
    code = (uint32_t)__builtin_rintf(a * 512.0f);
  } else {
    int E = (int)((__float_as_uint(a) >> 23) & 0xff) - 127;  // a is a normal fp32
    const uint32_t r = (uint32_t)__builtin_rintf(__builtin_ldexpf(a, 3 - E));  // 8 .. 16
    const bool carry = r == 16;
    E += carry ? 1 : 0;
    code = ((uint32_t)(E + 7) << 3) | (carry ? 0u : r - 8);
  }
  return code | sign;
}

// smallest e >= -127 with amax <= 448 * 2^e; 0 for amax = 0
__device__ __forceinline__ int act_exponent(float amax) {
  if (amax == 0.0f) return 0;
  if (amax < 0x1p-119f) return -127;  // exponent field <= -120: the floor
  const uint32_t b = __float_as_uint(amax);
  const int E = (int)((b >> 23) & 0xff) - 127;  // amax = (1 + f) 2^E, f < 1
  // amax 2^-(E-8) = (1 + f) 256 <= 448 iff 1 + f <= 1.75 (mantissa bits 0x600000)
  return (b & 0x7fffff) <= 0x600000u ? E - 8 : E - 7;
}

// Eight bf16 values (an uint4) to eight E4M3 bytes of v * 2^-e, |v| <= 448 *
// 2^e: gfx950's scaled conversion, which takes the scale 2^e itself. It gives
// e4m3_rne's byte for every bf16 value under every exponent -127 .. 120 that
// its block can have (tests/test_gpu_e4m3_conversions.py runs them all against the
// oracle's rounding, and samples of fp32 values through e4m3x8_of_f32).
__device__ __forceinline__ uint2 e4m3x8_of_bf16(uint4 w, int e) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  const float s = __builtin_ldexpf(1.0f, e);
  i16x2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, __builtin_bit_cast(bf16x2_t, w.x), s, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, __builtin_bit_cast(bf16x2_t, w.y), s, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(bf16x2_t, w.z), s, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(bf16x2_t, w.w), s, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
__device__ __forceinline__ uint2 e4m3x8_of_f32(const float (&v)[8], int e) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  const float s = __builtin_ldexpf(1.0f, e);
  i16x2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[0], v[1], s, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], s, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[4], v[5], s, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], s, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

// largest of eight 16-bit patterns (as unsigned numbers), and the largest
// magnitude among eight bf16 values as a pattern (0 .. 0x7fff)
__device__ __forceinline__ uint32_t bf16x8_max_bits(uint4 w) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const auto two = [](uint32_t v) { return __builtin_bit_cast(u16x2, v); };
  const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(two(w.x), two(w.y)),
                                            __builtin_elementwise_max(two(w.z), two(w.w)));
  return m[0] > m[1] ? m[0] : m[1];
}
__device__ __forceinline__ uint32_t bf16x8_max_abs(uint4 w) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return bf16x8_max_bits(make_uint4(w.x & kMag, w.y & kMag, w.z & kMag, w.w & kMag));
}

// n / d for 0 <= n < 2^31 by a multiplication: d > 1, made on the host
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv of(uint32_t d) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    return FastDiv{(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l - 1};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return __umulhi(n, mul) >> shift; }
};

// maximum over the 16 lanes of a DPP row, on every lane of the row
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t k) {
  k = max(k, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k, kDppXor1, 0xF, 0xF, false));
  k = max(k, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k, kDppXor2, 0xF, 0xF, false));
  k = max(k, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k, kDppHalfMirror, 0xF, 0xF, false));
  k = max(k, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k, kDppMirror, 0xF, 0xF, false));
  return k;
}

}  // namespace moe
