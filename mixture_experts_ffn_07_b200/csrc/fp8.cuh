// Block-scaled 8-bit floats: 128 values share one f32 scale.
//
// With a = max(max|x|, 2^-100) over the block and top the format's largest value (448 for e4m3, 57344 for
// e5m2): scale = a / top, inv = top / a, both rounded to f32, and code = the format's nearest value (half to
// even) of the f32 product x * inv.  With power-of-two scales: scale = 2^ceil(log2(a / top)), inv = 1 / scale,
// both exact.  The floor of 2^-100 keeps scale and inv finite and normal for blocks of zeros.  A NaN or an
// infinity in a block makes that block's values NaN (the maximum is taken on the bit patterns, where NaN is
// largest).
#pragma once

#include "kernels.h"

namespace moe {
namespace {

constexpr int kFp8Block = 128;

__device__ __forceinline__ float fp8_top(int fmt) { return fmt == MOE_E5M2 ? 57344.f : 448.f; }

// `amax_bits`: the largest |x| of the block as f32 bits.
__device__ __forceinline__ void fp8_scale(uint32_t amax_bits, int fmt, bool pow2, float& scale, float& inv) {
  const uint32_t floor_bits = (127u - 100u) << 23;
  const uint32_t b = amax_bits > floor_bits ? amax_bits : floor_bits;
  const float a = __uint_as_float(b);
  if (pow2) {
    // a = m 2^e, top = 1.75 2^t with t = 8 or 15: a / top = (m / 1.75) 2^(e - t), so ceil(log2) is e - t for
    // m <= 1.75 and e - t + 1 above
    const int t = fmt == MOE_E5M2 ? 15 : 8;
    const int e = static_cast<int>(b >> 23) - t + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    scale = (b >> 23) == 255u ? a : __uint_as_float(static_cast<uint32_t>(e) << 23);
    inv = (b >> 23) == 255u ? (a != a ? a : 0.f) : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  } else {
    scale = __fdiv_rn(a, fp8_top(fmt));
    inv = __fdiv_rn(fp8_top(fmt), a);
  }
}

// Codes of two values: the first in the low byte.
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi, int fmt) {
  uint16_t r;
  if (fmt == MOE_E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace
}  // namespace moe
