// act_q8.h -- the 8-bit quantization of activations that the W4A8 linears and
// the RMS norm in front of them share: symmetric, one scale per row or per
// group of 32, scales and codes in binary32.  Internal header.
#pragma once

#include "qg_common.h"

namespace qg {

// The absmax keeps a NaN: nmax is the IEEE 754-2019 maximum (one
// v_maximum3_f32 on gfx950), which returns NaN when either input is NaN,
// where fmaxf would return the other input.  An infinity survives any max.
__device__ __forceinline__ float nmax(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A span whose absmax is not finite (it holds a NaN or an infinity) has no
// finite scale: its absmax becomes NaN, which gives inv = 0 through
// a > 0 ? 127 / a : 0 and sx = a / 127 = NaN, so every output the span
// reaches is NaN.
__device__ __forceinline__ float finite_or_nan(float a) {
  return a < __builtin_inff() ? a : __builtin_nanf("");
}

// The span's scales from its absmax a (>= 0, or NaN as above): inv = 127 / a
// and sx = a / 127, both correctly rounded binary32 divisions.  Where 127 / a
// is not a finite binary32 number there is no inverse scale and inv = 0, so
// every code is 0: for a == 0 and for a span so small that the quotient
// overflows (a <= 127 * 2^-128), sx = 0 as well (a zero span, outputs 0); for
// a NaN absmax sx stays NaN.
__device__ __forceinline__ void span_scale(float a, float& inv, float& sx) {
  inv = 127.0f / a;
  sx = a / 127.0f;
  if (!(inv <= __FLT_MAX__)) {
    inv = 0.0f;
    if (a == a) sx = 0.0f;
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_fa(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                               CTRL, 0xf, 0xf, true));
}

}  // namespace qg
