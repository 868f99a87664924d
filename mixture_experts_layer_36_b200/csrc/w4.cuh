// The 4-bit weight format (include/moe.h, "4-bit expert weights"): the scale and
// code rules.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

// s = bf16(max / 7), 1 where that is 0.  max has 8 significant bits: max / 7 is
// a bf16 value or at least 2^-12 of itself away from where bf16 rounding turns,
// so a product that is 2^-23 off rounds to the same.
__device__ __forceinline__ __nv_bfloat16 w4_scale(float mx) {
  const __nv_bfloat16 s = __float2bfloat16(mx * (1.0f / 7.0f));
  return __bfloat162float(s) == 0.f ? __float2bfloat16(1.0f) : s;
}

// u = 8 + rne(v / s) in 1..15; 8 where the scale is not finite (an infinity or
// a NaN in the group), which then reads back as 0 * inf = NaN.
__device__ __forceinline__ uint32_t w4_code(float v, float s) {
  const float r = rintf(__fdiv_rn(v, s));
  const int c = (fabsf(s) <= 3.4e38f) ? max(-7, min(7, static_cast<int>(r))) : 0;
  return static_cast<uint32_t>(c + 8);
}

// The same without a division, for scales in [2^-120, 2^120], as the bits of
// kW4Bits + u: v / s is a half-integer or, both having 8 significant bits, at
// least 1/510 away from one, so v * inv (1e-6 off) rounded to a multiple of 2^-10
// (by the first addend's unit) is on the half-integer or on the right side of it,
// and the second addend rounds that to an integer, halves to even.  Up to 7.03,
// which needs no clamp: s is 7.03 or less of the largest value's 1/7 there.
constexpr float kW4Step = 12288.0f;                       // 1.5 2^13
constexpr uint32_t kW4Bits = 0x4B400000u;                 // of 1.5 2^23
__device__ __forceinline__ uint32_t w4_code_bits(float v, float inv) {
  return __float_as_uint(fmaf(v, inv, kW4Step) + (12582912.0f + 8.0f - kW4Step));
}
__device__ __forceinline__ bool w4_scale_plain(float s) { return s >= 7.5e-37f && s <= 1.3e36f; }

}  // namespace moe
