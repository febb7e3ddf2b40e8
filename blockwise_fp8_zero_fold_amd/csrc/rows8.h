// Rows in 8 bits: E4M3 codes with one scale per group of 128 columns.  The group's scale is
// amax / 448 (or the power of two 2^(floor(log2 amax) - 8)) as the blocks of the weights have it, and
// 1 for a group of zeros; not below 2^-126, so that dividing by it never overflows what is finite.
// A code is x / scale rounded to nearest, ties to even, and saturated at 448; NaN stays NaN, and so do the
// infinities of a group that holds one (inf / inf; the group's other codes are 0, and stand for 0 * inf).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace fp8z1 {

constexpr float kTop8 = 448.0f;  // largest E4M3 value

__device__ __forceinline__ float row8_scale(float amax, bool pow2) {
  if (amax == 0.0f) return 1.0f;
  float s = amax / kTop8;
  if (pow2) {
    // the exponent's field less 8 (of a subnormal amax the least there is; an infinite amax stays so)
    const int32_t e = static_cast<int32_t>(__float_as_uint(amax) >> 23) - 8;
    if (amax < __builtin_huge_valf()) s = __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
  }
  return fmaxf(s, 0x1p-126f);
}

// Division by a group's scale: Markstein's correctly rounded division (Computation of elementary functions on the IBM RISC
// System/6000 processor, IBM Journal of Research and Development 34, 1990), a reciprocal refined once and a
// quotient corrected twice by its remainder, with the reciprocal taken once for the group.  For scales from 2^-60 to
// 2^60 nothing in them leaves the normal numbers unless the quotient is below 2^-20, which is code 0 either way; other
// scales are brought there by a power of two, and so is what is divided (`times`; what that takes below the normal
// numbers has a quotient below 2^-120).  Of an infinite scale, times is 0 and the scale 1: 0 of what is finite.
struct Over8 {
  float scale, inverse, times;
};
__device__ __forceinline__ Over8 over8(float scale) {
  float times = 1.0f;
  if (scale < 0x1p-60f) times = 0x1p66f;
  if (scale > 0x1p60f) times = 0x1p-66f;
  float s = scale * times;
  if (scale == __builtin_huge_valf()) s = 1.0f, times = 0.0f;
  const float r = __builtin_amdgcn_rcpf(s);
  return Over8{s, fmaf(fmaf(-s, r, 1.0f), r, r), times};
}

// 4 values over their group's scale as codes, the first in the lowest byte.  The hardware's conversion rounds to
// nearest even; what it makes of values past 448 (which the rule of powers of two has) hangs on a mode, so they are
// cut off before it.  The sign is x's own, since a zero loses its sign in the sums.
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, const Over8& o) {
  auto over = [&](float v) {
    const float x = v * o.times;
    const float q0 = x * o.inverse, q1 = fmaf(fmaf(-q0, o.scale, x), o.inverse, q0);
    const float q = fmaf(fmaf(-q1, o.scale, x), o.inverse, q1);
    return copysignf(fabsf(q) > kTop8 ? kTop8 : q, v);
  };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(over(x0), over(x1), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(over(x2), over(x3), w, true);
  return static_cast<uint32_t>(w);
}

}  // namespace fp8z1
