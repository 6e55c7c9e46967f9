// wave.h -- sums, maxima and running sums over the 64 lanes of a wave in
// registers (DPP moves, no LDS).  Internal header.
#pragma once

#include "qg_common.h"

namespace qg {

// v of the lane that a DPP control names; `none` where it names none, or where the
// row is masked out.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or(uint32_t v, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float v, float none) {
  return __uint_as_float(dpp_or<CTRL, ROWS>(__float_as_uint(v), __float_as_uint(none)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp_or(uint64_t v, uint64_t none) {
  return (uint64_t)dpp_or<CTRL, ROWS>((uint32_t)(v >> 32), (uint32_t)(none >> 32)) << 32 |
         dpp_or<CTRL, ROWS>((uint32_t)v, (uint32_t)none);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or(double v, double none) {
  return __longlong_as_double((long long)dpp_or<CTRL, ROWS>((uint64_t)__double_as_longlong(v),
                                                            (uint64_t)__double_as_longlong(none)));
}

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); }
__device__ __forceinline__ float lane_of(float v, int l) { return __uint_as_float(lane_of(__float_as_uint(v), l)); }
__device__ __forceinline__ uint64_t lane_of(uint64_t v, int l) {
  return (uint64_t)lane_of((uint32_t)(v >> 32), l) << 32 | lane_of((uint32_t)v, l);
}
__device__ __forceinline__ double lane_of(double v, int l) {
  return __longlong_as_double((long long)lane_of((uint64_t)__double_as_longlong(v), l));
}

// v joined with all lanes before it, by an operation whose neutral element is `none`.
template <class T, class Op>
__device__ __forceinline__ T wave_scan(T v, T none, Op op) {
  v = op(v, dpp_or<0x111, 0xf>(v, none));   // row_shr 1, 2, 4, 8
  v = op(v, dpp_or<0x112, 0xf>(v, none));
  v = op(v, dpp_or<0x114, 0xf>(v, none));
  v = op(v, dpp_or<0x118, 0xf>(v, none));
  v = op(v, dpp_or<0x142, 0xa>(v, none));   // row_bcast 15, 31
  v = op(v, dpp_or<0x143, 0xc>(v, none));
  return v;
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {   // the same in all lanes
  return lane_of(wave_scan(v, T(0), [](T a, T b) { return a + b; }), 63);
}

__device__ __forceinline__ float wave_max(float v) {   // of numbers; a NaN gives way
  return lane_of(wave_scan(v, -__builtin_inff(), [](float a, float b) { return fmaxf(a, b); }), 63);
}

// The running sum before this lane; `all`: over all.
__device__ __forceinline__ uint64_t wave_before(uint64_t mine, uint64_t& all) {
  const uint64_t sum = wave_scan(mine, (uint64_t)0, [](uint64_t a, uint64_t b) { return a + b; });
  all = lane_of(sum, 63);
  return sum - mine;
}

}  // namespace qg
