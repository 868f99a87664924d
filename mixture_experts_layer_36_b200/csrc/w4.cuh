// The 4-bit weight format (include/moe.h, "4-bit expert weights"): the scale and
// code rules.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

// s = bf16(max / 7), 1 where that is 0.  __fdiv_rn: the bf16 maximum has 8
// significant bits, so the fp32 quotient is never close enough to a bf16
// rounding border for its own rounding to matter.
__device__ __forceinline__ __nv_bfloat16 w4_scale(float mx) {
  const __nv_bfloat16 s = __float2bfloat16(__fdiv_rn(mx, 7.0f));
  return __bfloat162float(s) == 0.f ? __float2bfloat16(1.0f) : s;
}

// u = 8 + rne(v / s) in 1..15; 8 where v / s is not finite (an infinity or a
// NaN in the group: its scale is not finite, so any code reads back as NaN
// only if it is 8, 0 * inf)
__device__ __forceinline__ uint32_t w4_code(float v, float s) {
  const float r = rintf(__fdiv_rn(v, s));
  const int c = (fabsf(s) <= 3.4e38f) ? max(-7, min(7, static_cast<int>(r))) : 0;
  return static_cast<uint32_t>(c + 8);
}

}  // namespace moe
