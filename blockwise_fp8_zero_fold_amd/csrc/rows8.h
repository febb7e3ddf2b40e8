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
    // the exponent's field less 8; (of an infinite amax the largest power there is, of a subnormal the least)
    const int32_t e = static_cast<int32_t>(__float_as_uint(amax) >> 23) - 8;
    if (amax < __builtin_huge_valf()) s = __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
  }
  return fmaxf(s, 0x1p-126f);
}

// Division by a group's scale.  The steps are those of a correctly rounded division (a reciprocal refined once, a
// quotient corrected twice by its remainder), with the reciprocal taken once for the group and no scaling of the
// operands: for scales from 2^-60 to 2^60 nothing in them leaves the normal numbers unless the quotient is below
// 2^-20, which is code 0 either way.
struct Over8 {
  float scale, inverse;
  bool plain;  // scales outside that range: a division each
  bool cut;    // the power of two rule, whose quotients may pass 448
};
__device__ __forceinline__ Over8 over8(float scale, bool pow2) {
  const float r = __builtin_amdgcn_rcpf(scale);
  return Over8{scale, fmaf(fmaf(-scale, r, 1.0f), r, r), !(scale >= 0x1p-60f && scale <= 0x1p60f), pow2};
}
__device__ __forceinline__ float quotient8(float x, const Over8& o) {
  if (o.plain) return x / o.scale;
  const float q0 = x * o.inverse, q1 = fmaf(fmaf(-q0, o.scale, x), o.inverse, q0);
  return copysignf(fmaf(fmaf(-q1, o.scale, x), o.inverse, q1), x);  // (a zero's sign is lost in the sums)
}

// 4 values over their group's scale as codes, the first in the lowest byte.  The hardware's conversion rounds to
// nearest even; what it makes of values past 448 hangs on a mode, so they are cut off before it.
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, const Over8& o) {
  auto over = [&](float x) {
    const float q = quotient8(x, o);
    if (!o.cut) return q;  // (amax / (amax / 448) rounds to 448 or its neighbours, which are code 448)
    const float c = fminf(fmaxf(q, -kTop8), kTop8);
    return q != q ? q : c;
  };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(over(x0), over(x1), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(over(x2), over(x3), w, true);
  return static_cast<uint32_t>(w);
}

}  // namespace fp8z1
