// qk_norm_rope.hip -- RMS norm of every query and key head and the rotation
// of its channels by position, in one pass (qg_qk_norm_rope).
//
//   y = x * rsqrt(mean(x^2) + eps) * w               per head of d channels
//   (a, b) -> (a cos - b sin, b cos + a sin)         the first `rot` channels
// in fp32, rounded once to bf16.
//
// Mapping: a lane owns 16 channels of a head, chosen so that both members of
// a rotated pair are its own (halves: channels 8j.. and rot/2 + 8j..;
// adjacent pairs: 16j..), so the rotation needs no cross-lane move and the sum
// of squares is a butterfly over the head's lanes (d / 16 of them, padded to a
// power of two).  A wave takes 64 / lanes heads of one token at a time and
// walks `iters` such groups, keeping the token's cos and sin (the same channel
// pairs for every head) in registers: read once per token and wave rather than
// once per head, they are 1/40 of the traffic at 40 heads of 128.
//
// Bound by HBM for long inputs (2 bytes read and 2 written per channel): 16383
// tokens of 32 + 8 heads of 128, 344 MB, take 68.5 us or 5.0 TB/s, what a large
// copy reaches (5.1).  A decode step is bound by its launch: 2.8 us for 1 token,
// 3.2 us for 61 tokens of 16 + 2 heads of 256.
#include "qg_common.h"
#include "layer_common.h"

namespace qg {

// x[16] of one lane as fp32 from two 16-byte loads.
__device__ __forceinline__ void unpack8(const u32x4_t& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

template <int LPH>   // lanes per head, a power of two
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(NormRopeArgs a) {
  constexpr int SLOTS = 64 / LPH;
  const int lane = threadIdx.x & 63;
  const int j = lane % LPH, slot = lane / LPH;
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave_id_uniform();
  const int64_t t = unit / a.chunks;
  if (t >= a.tokens) return;
  const int h0 = (int)(unit - t * a.chunks) * SLOTS * a.iters + slot;
  const int heads = a.hq + a.hkv;
  const bool live = 16 * j < a.d;
  const bool turned = 16 * j < a.rot;
  // channels of this lane: [c0, c0 + 8) and [c1, c1 + 8)
  const bool halves = turned && !a.pairs;
  const int c0 = halves ? 8 * j : 16 * j;
  const int c1 = halves ? a.rot / 2 + 8 * j : 16 * j + 8;

  // A position outside the table reads row 0 and turns the token's heads into NaN.
  const int pos = a.positions[t];
  const bool bad = pos < 0 || pos >= a.max_pos;
  float cs[8], sn[8];
  if (turned) {
    const float* row = a.cos_sin + (size_t)(bad ? 0 : pos) * a.rot + 8 * j;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t c = *reinterpret_cast<const f32x4_t*>(row + 4 * i);
      const f32x4_t s = *reinterpret_cast<const f32x4_t*>(row + a.rot / 2 + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[4 * i + e] = c[e];
        sn[4 * i + e] = s[e];
      }
    }
  }
  if (bad && a.status && lane == 0) atomicOr(a.status, QG_FLAG_POSITION);

  for (int it = 0; it < a.iters; ++it) {
    const int h = h0 + it * SLOTS;
    const bool on = live && h < heads;
    const bool is_q = h < a.hq;
    const int hh = is_q ? h : h - a.hq;
    u32x4_t v0{}, v1{}, w0, w1;
    const uint16_t* const w = is_q ? a.qw : a.kw;
    w0 = w1 = u32x4_t{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};   // no weight: ones
    if (on) {
      const uint16_t* x = is_q ? a.q + t * a.q_ts + hh * a.q_hs : a.k + t * a.k_ts + hh * a.k_hs;
      v0 = *reinterpret_cast<const u32x4_t*>(x + c0);
      v1 = *reinterpret_cast<const u32x4_t*>(x + c1);
      if (w) {
        w0 = *reinterpret_cast<const u32x4_t*>(w + c0);
        w1 = *reinterpret_cast<const u32x4_t*>(w + c1);
      }
    }
    float x0[8], x1[8], g0[8], g1[8];
    unpack8(v0, x0);
    unpack8(v1, x1);
    unpack8(w0, g0);
    unpack8(w1, g1);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss = __builtin_fmaf(x0[e], x0[e], ss);
      ss = __builtin_fmaf(x1[e], x1[e], ss);
    }
#pragma unroll
    for (int o = 1; o < LPH; o *= 2) ss += __shfl_xor(ss, o);
    const float mean = ss * a.inv_d + a.eps;
    float r = 1.0f / sqrtf(mean);
    // Channels from 2^63 on, and small ones where eps is no larger: their squares leave
    // binary32, so such heads are taken times 2^-72 or 2^72, which the norm takes off again.
    const float c = ss == __builtin_inff() ? 0x1p-72f : mean < 0x1p-90f ? 0x1p72f : 1.0f;
    if (__ballot(c != 1.0f) != 0) {
      ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x0[e] *= c;
        x1[e] *= c;
        ss = __builtin_fmaf(x0[e], x0[e], ss);
        ss = __builtin_fmaf(x1[e], x1[e], ss);
      }
#pragma unroll
      for (int o = 1; o < LPH; o *= 2) ss += __shfl_xor(ss, o);
      r = 1.0f / sqrtf(ss * a.inv_d + a.eps * c * c);
    }
    if (bad) r = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x0[e] = x0[e] * r * g0[e];
      x1[e] = x1[e] * r * g1[e];
    }
    if (turned) {
      if (a.pairs) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = x0[2 * e], q = x0[2 * e + 1], u = x1[2 * e], z = x1[2 * e + 1];
          x0[2 * e] = p * cs[e] - q * sn[e];
          x0[2 * e + 1] = q * cs[e] + p * sn[e];
          x1[2 * e] = u * cs[4 + e] - z * sn[4 + e];
          x1[2 * e + 1] = z * cs[4 + e] + u * sn[4 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = x0[e], q = x1[e];
          x0[e] = p * cs[e] - q * sn[e];
          x1[e] = q * cs[e] + p * sn[e];
        }
      }
    }
    if (on) {
      uint16_t* y = is_q ? a.q_out + ((size_t)t * a.hq + hh) * a.d : a.k_out + ((size_t)t * a.hkv + hh) * a.d;
      u32x4_t o0, o1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o0[e] = pack_bf16(x0[2 * e], x0[2 * e + 1]);
        o1[e] = pack_bf16(x1[2 * e], x1[2 * e + 1]);
      }
      *reinterpret_cast<u32x4_t*>(y + c0) = o0;
      *reinterpret_cast<u32x4_t*>(y + c1) = o1;
    }
  }
}

hipError_t launch_qk_norm_rope(NormRopeArgs a, hipStream_t stream) {
  int lph = 1;
  while (16 * lph < a.d) lph *= 2;
  const int slots = 64 / lph, heads = a.hq + a.hkv;
  const int groups = (heads + slots - 1) / slots;
  // One group of heads per wave while that gives no more than 16 waves per CU
  // (a decode batch: shortest chain of loads); whole tokens per wave above.
  a.iters = a.tokens * groups <= kCUs * 16 ? 1 : groups;
  a.chunks = (groups + a.iters - 1) / a.iters;
  const int64_t blocks = (a.tokens * a.chunks + 3) / 4;
#define QG_NR(L) \
  case L: hipLaunchKernelGGL((qk_norm_rope_kernel<L>), dim3((uint32_t)blocks), dim3(256), 0, stream, a); break;
  switch (lph) {
    QG_NR(1) QG_NR(2) QG_NR(4) QG_NR(8) QG_NR(16) QG_NR(32)
    default: return hipErrorInvalidValue;
  }
#undef QG_NR
  return hipGetLastError();
}

}  // namespace qg
