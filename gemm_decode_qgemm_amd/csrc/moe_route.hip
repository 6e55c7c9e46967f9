// moe_route.hip -- the choice of experts from a router's logits (qg_moe_route).
//
//   s = softmax(l) or sigmoid(l);   c = s + bias      (the bias decides, it does not weigh)
//   experts in equal groups: a group counts the sum of its best one or two c; the
//   best groups stay;   the top k experts by c among them, ties to the lowest index;
//   w = s of the picked, over their sum where renormalized, times a scale
//
// A wave takes a token, lane l experts U l .. U l + U - 1.  Which of two experts comes
// first is a comparison of computed numbers, and in 32 bits one choice in some
// thousands would go by rounding.  So:
//  * where no bias and no sum of two takes part, the order is that of the logits,
//    which are compared as they are;
//  * else c is formed in 32 bits with a bound on its error, and where all
//    numbers that were compared are further apart than that, the choice is the
//    exact one; a token where they are not (about one in a thousand) is done again
//    in 64 bits;
//  * groups that are not a power of two of whole lanes (160 and 384 experts in 2, 4 or 8,
//    for example) are chosen in 64 bits for every token, the logits alone among them
//    (us, 160 and 384 experts in 8 groups, against 128 and 512: one token 7.2, 10.1 / 3.3,
//    4.1; 61 8.8, 13.1 / 4.3, 5.8; 16385 37.7, 64.4 / 9.6, 23.9).
// Weights are formed in 64 bits from the picked logits, a lane each, by one wave for
// several tokens.
//
// The k-th largest c is found by bisection: a ballot per register and step, from
// the largest c down until exactly k are left above, about ten steps.
#include "layer_common.h"
#include "wave.h"

namespace qg {

// A number as an unsigned one of the same order; NaN is above all, -0 is 0, and none is 0.
__device__ __forceinline__ uint64_t order64(double c) {
  c += 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(c);
  if (c != c) return ~(uint64_t)0;
  return (u >> 63) != 0 ? ~u : u | (uint64_t)1 << 63;
}

__device__ __forceinline__ double from64(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) != 0 ? k ^ (uint64_t)1 << 63 : ~k));
}

// The same order for binary32 numbers, as steps of a bisection; and back.
__device__ __forceinline__ uint32_t step_of(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float step_to(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// The value of lane l ^ O, where lanes of an O-aligned block hold the same value.
template <int O>
__device__ __forceinline__ float other_block(float v) {
  if constexpr (O == 1) return dpp_f<0xB1>(v);         // quad_perm [1,0,3,2]
  if constexpr (O == 2) return dpp_f<0x4E>(v);         // quad_perm [2,3,0,1]
  if constexpr (O == 4) return dpp_f<0x141>(v);        // row_half_mirror
  if constexpr (O == 8) return dpp_f<0x140>(v);        // row_mirror
  return __shfl_xor(v, O);
}

// The best two over blocks of 2 O lanes from those of O.
template <int O>
__device__ __forceinline__ void best_two(int lanes, float& c1, float& c2) {
  if (O >= lanes) return;              // uniform
  const float d1 = other_block<O>(c1), d2 = other_block<O>(c2);
  c2 = fmaxf(fminf(c1, d1), fmaxf(c2, d2));
  c1 = fmaxf(c1, d1);
}

// A wave's own LDS: its operations complete in order.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct __attribute__((aligned(16))) Pick {
  float c, x;                          // what decides, and the logit
  int id, pad;
};

constexpr int kRouteTokens = 8;        // of a workgroup, a wave each

template <int U>
struct RouteLds {
  union {
    uint64_t choice[64 * U];           // of the exact way: every expert's key
    Pick by_expert[32];
  };
};

// U values from the lane's place on in a row of n, `none` past it.  `whole`: rows and
// places are aligned to U values, and n is a multiple of U.
template <int U>
__device__ __forceinline__ void load_row(float (&v)[U], const void* row, bool half, bool whole, int n, float none) {
  const int e = U * (int)(threadIdx.x & 63);
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = none;
  if (whole) {
    if (e >= n) return;
    if (half) {
      struct __attribute__((aligned(2 * U))) Pack { uint16_t v[U]; };
      const Pack p = *reinterpret_cast<const Pack*>(static_cast<const uint16_t*>(row) + e);
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = bf16_to_f32(p.v[u]);
    } else {
      struct __attribute__((aligned(U < 4 ? 4 * U : 16))) Pack { float v[U]; };
      const Pack p = *reinterpret_cast<const Pack*>(static_cast<const float*>(row) + e);
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = p.v[u];
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e + u < n) v[u] = half ? bf16_to_f32(static_cast<const uint16_t*>(row)[e + u]) : static_cast<const float*>(row)[e + u];
  }
}

// exp(x - top) in 64 bits; 0 for -infinity (a token without a logit above it has no
// scores), and none beside an infinite one.
__device__ __forceinline__ double route_exp(float x, float top) {
  const double d = top == __builtin_inff() ? (double)__builtin_nanf("") : (double)x - (double)top;
  return x == -__builtin_inff() && !(top == __builtin_inff()) ? 0.0 : exp(d);
}

template <int U>
__device__ __forceinline__ double route_total(const float (&l)[U], float top) {
  double total = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u) total += route_exp(l[u], top);
  return wave_sum(total);
}

template <int O>
__device__ __forceinline__ uint64_t other_block64(uint64_t v) {
  return (uint64_t)__float_as_uint(other_block<O>(__uint_as_float((uint32_t)(v >> 32)))) << 32 |
         __float_as_uint(other_block<O>(__uint_as_float((uint32_t)v)));
}
template <int O>
__device__ __forceinline__ void best_two64(int lanes, uint64_t& k1, uint64_t& k2) {
  if (O >= lanes) return;              // uniform
  const uint64_t d1 = other_block64<O>(k1), d2 = other_block64<O>(k2);
  k2 = max(min(k1, d1), max(k2, d2));
  k1 = max(k1, d1);
}

// The whole choice in 64 bits: lane j's pick.  By k rounds: the largest key of the
// wave, then the lowest expert that has it.
template <int U>
__device__ __forceinline__ int route_exact(const RouteArgs& a, const float (&l)[U], float top, RouteLds<U>& lds) {
  const int lane = threadIdx.x & 63;
  uint64_t key[U];
  const bool by_logit = a.bias == nullptr && (a.groups == 1 || a.best == 1);
  const double total = by_logit || a.sigmoid ? 0.0 : route_total(l, top);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = U * lane + u;
    double c = (double)l[u];
    if (!by_logit) {
      if (a.sigmoid)
        c = 1.0 / (1.0 + exp(-c));
      else
        c = total == 0.0 ? 0.0 : route_exp(l[u], top) / total;
      if (a.bias && e < a.e) c += (double)a.bias[e];
    }
    key[u] = e < a.e ? order64(c) : 0;
  }
  if (a.groups > 1 && a.lanes > 0) {   // groups of whole lanes
    uint64_t k1 = key[0], k2 = 0;      // the best two of this lane, then of the group
#pragma unroll
    for (int u = 1; u < U; ++u) {
      k2 = max(min(k1, key[u]), k2);
      k1 = max(k1, key[u]);
    }
    best_two64<1>(a.lanes, k1, k2);
    best_two64<2>(a.lanes, k1, k2);
    best_two64<4>(a.lanes, k1, k2);
    best_two64<8>(a.lanes, k1, k2);
    best_two64<16>(a.lanes, k1, k2);
    best_two64<32>(a.lanes, k1, k2);
    const uint64_t value = a.best == 1 ? k1 : order64(from64(k1) + from64(k2));
    const int own = lane >> a.shift;
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t other = lane_of(value, g << a.shift);
      before += other > value || (other == value && g < own);
    }
    if (before >= a.top_groups)
#pragma unroll
      for (int u = 0; u < U; ++u) key[u] = 0;
  } else if (a.groups > 1) {
#pragma unroll
    for (int u = 0; u < U; ++u) lds.choice[U * lane + u] = key[u];
    wave_fence();
    const int per = a.e / a.groups;
    uint64_t k1 = 0, k2 = 0;           // lane g: the best two of group g
    if (lane < a.groups)
      for (int i = 0; i < per; ++i) {
        const uint64_t k = lds.choice[lane * per + i];
        k2 = max(min(k1, k), k2);
        k1 = max(k1, k);
      }
    const uint64_t mine = lane >= a.groups ? 0 : a.best == 1 ? k1 : order64(from64(k1) + from64(k2));
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t other = lane_of(mine, g);
      before += other > mine || (other == mine && g < lane);
    }
    const uint64_t open = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((open >> ((U * lane + u) / per & 63) & 1) == 0) key[u] = 0;
  }
  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t m = key[0];
#pragma unroll
    for (int u = 1; u < U; ++u) m = max(m, key[u]);
    const auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
    const uint32_t hi = lane_of(wave_scan((uint32_t)(m >> 32), 0u, larger), 63);
    const uint32_t lo = lane_of(wave_scan((uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u, 0u, larger), 63);
    m = (uint64_t)hi << 32 | lo;
    int first = U;                     // of this lane's experts that have it
#pragma unroll
    for (int u = U - 1; u >= 0; --u)
      if (key[u] == m) first = u;
    const int at = __builtin_ctzll(__ballot(first < U));
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane == at && u == first) key[u] = 0;
    const int e = U * at + __builtin_amdgcn_readlane(first, at);
    if (lane == j) id = e;
  }
  return id;
}

template <int U>
__device__ __forceinline__ int count_from(const float (&c)[U], float from) {
  int n = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) n += __popcll(__ballot(c[u] >= from));
  return n;
}

// Bits of the mask below this lane, added to n.
__device__ __forceinline__ int bits_below(uint64_t mask, int n) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, n));
}

// A token's picks in order, `to`[0 .. k - 1], by a wave.
template <int U>
__device__ __forceinline__ void route_token(const RouteArgs& a, const float (&l)[U], const float (&b)[U], float top,
                                            RouteLds<U>& lds, int* id_to, float* x_to) {
  const int lane = threadIdx.x & 63;
  // c as binary32, off by at most `off`.  Sigmoid: an exponential is off by 2^-23 of
  // itself and what the rounding of its argument adds, |l| 2^-24, of which s (1 - s) < 1/4
  // and s (1 - s) |l| < 0.3 counts; a reciprocal by 2^-23: 2^-22 in all.  Softmax: likewise
  // 2^-23 + 2.5 x 2^-24 of e^-x with x e^-x < 0.4, and the sum, up to 40 additions of
  // 2^-24 one after another: 2^-18.5 of the largest score.  The last addition: 2^-24 of c.
  const bool exact = a.bias == nullptr && (a.groups == 1 || a.best == 1);
  float c[U];
  float most = 1.0f;                   // the largest score, at most
#pragma unroll
  for (int u = 0; u < U; ++u) c[u] = l[u];
  if (!exact) {
    constexpr float kLog2e = 1.44269504088896340736f;
    if (a.sigmoid) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        c[u] = b[u] + __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[u]));
    } else {
      float total = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        c[u] = l[u] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(kLog2e * (l[u] - top));
        total += c[u];
      }
      total = wave_sum(total);
      most = total == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = b[u] + c[u] * most;
    }
  }
  const float least = a.sigmoid ? 0x1p-21f : most * 0x1p-18f;
  auto off = [&](float v) { return __builtin_fmaf(fabsf(v), 0x1p-23f, least); };
  bool near = false;                   // numbers that 32 bits do not tell apart, or a NaN
#pragma unroll
  for (int u = 0; u < U; ++u) near |= c[u] != c[u] && U * lane + u < a.e;
  // From here on a NaN is an expert that is not there: no comparison holds.
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (U * lane + u >= a.e) c[u] = __builtin_nanf("");

  if (a.groups > 1) {
    near |= a.lanes == 0;
    const int lanes = max(a.lanes, 1);
    float c1 = c[0], c2 = -__builtin_inff();   // the best two of this lane, then of the group
#pragma unroll
    for (int u = 1; u < U; ++u) {
      c2 = fmaxf(fminf(c1, c[u]), c2);
      c1 = fmaxf(c1, c[u]);
    }
    best_two<1>(lanes, c1, c2);
    best_two<2>(lanes, c1, c2);
    best_two<4>(lanes, c1, c2);
    best_two<8>(lanes, c1, c2);
    best_two<16>(lanes, c1, c2);
    best_two<32>(lanes, c1, c2);
    const float value = a.best == 1 ? c1 : c1 + c2;
    const int own = lane >> a.shift, first = lane & (lanes - 1);
    float n = 0.0f;                    // groups before this one
    // A group's lanes compare it with one other group each, in turn.
    for (int g0 = 0; g0 < a.groups; g0 += lanes) {
      const int g = g0 + first;
      const float other = __shfl(value, min(g, a.groups - 1) << a.shift);
      const bool is = g < a.groups && own < a.groups && g != own;
      n += is && (other > value || (other == value && g < own)) ? 1.0f : 0.0f;
    }
    if (lanes > 1) n += other_block<1>(n);
    if (lanes > 2) n += other_block<2>(n);
    if (lanes > 4) n += other_block<4>(n);
    if (lanes > 8) n += other_block<8>(n);
    if (lanes > 16) n += other_block<16>(n);
    if (lanes > 32) n += other_block<32>(n);
    const bool stay = own < a.groups && n < (float)a.top_groups;
    if (!exact) {                      // the last group that stays and the first that does not
      const float e = 1.5f * (off(c1) + off(a.best == 1 ? c1 : c2));
      const float stays = -wave_max(stay ? e - value : -__builtin_inff());
      const float goes = wave_max(own < a.groups && !stay ? value + e : -__builtin_inff());
      near |= !(stays > goes);
    }
    if (!stay)
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = __builtin_nanf("");
  }

  bool sure = __ballot(near) == 0;
  if (sure) {
    float high = c[0];
#pragma unroll
    for (int u = 1; u < U; ++u) high = fmaxf(high, c[u]);
    high = wave_max(high);
    // From the largest down in strides until k are reached, then by halves: k or more
    // from `lo` on, fewer from `hi` on.
    const uint32_t lowest = step_of(-__builtin_inff());
    uint32_t hi = step_of(high) + 1u, lo = hi;
    int n = 0;
    for (uint32_t d = 1u << 21; n < a.k; d <<= 2) {
      hi = lo;
      lo = lo - lowest > d && d != 0u ? lo - d : lowest;
      n = count_from(c, step_to(lo));
      if (lo == lowest) break;
    }
    while (n != a.k && hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int m = count_from(c, step_to(mid));
      if (m >= a.k)
        lo = mid, n = m;
      else
        hi = mid;
    }
    const float from = step_to(lo);
    bool mine[U];
#pragma unroll
    for (int u = 0; u < U; ++u) mine[u] = c[u] >= from;
    if (n != a.k) {                    // several that are equal: of those the lowest, as many as are left
      int left = a.k, before = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) left -= __popcll(__ballot(c[u] > from));
#pragma unroll
      for (int u = 0; u < U; ++u) before = bits_below(__ballot(c[u] == from), before);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c[u] == from) mine[u] = before++ < left;
    }
    int place = 0;                     // among the picks, in order of experts
#pragma unroll
    for (int u = 0; u < U; ++u) place = bits_below(__ballot(mine[u]), place);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (mine[u]) lds.by_expert[place++] = Pick{c[u], l[u], U * lane + u, 0};
    wave_fence();
    // Every pick against every other: 64 / `room` lanes a pick, one other each in turn.
    const int room = a.k <= 8 ? 8 : a.k <= 16 ? 16 : 32, turn = 64 / room, at = lane / turn;
    const Pick p = lds.by_expert[at];
    const float far = 2.0f * off(p.c);
    float rank = 0.0f;
    for (int j = lane & (turn - 1); j < room; j += turn) {
      const float other = lds.by_expert[j].c;
      const bool is = j < a.k && at < a.k && j != at;
      rank += is && (other > p.c || (other == p.c && j < at)) ? 1.0f : 0.0f;
      if (!exact) near |= is && !(fabsf(other - p.c) > far);
    }
    rank += other_block<1>(rank);
    if (turn > 2) rank += other_block<2>(rank);
    if (turn > 4) rank += other_block<4>(rank);
    if (!exact) {                      // and the last pick against the first that is none
      const uint64_t last = __ballot(at < a.k && rank == (float)(a.k - 1));
      const float v = lane_of(p.c, last != 0 ? __builtin_ctzll(last) : 0);
      near |= count_from(c, __builtin_fmaf(-2.5f, off(v), v)) != a.k;
      sure = __ballot(near) == 0;
    }
    if (sure && at < a.k && (lane & (turn - 1)) == 0) id_to[(int)rank] = p.id, x_to[(int)rank] = p.x;
  }
  if (!sure) {
    wave_fence();
    const int id = route_exact(a, l, top, lds);
    if (lane >= a.k) return;
    id_to[lane] = id;
    // out of the registers of the lane that has it, by way of LDS, would take longer
    const size_t at = (size_t)((int64_t)blockIdx.x * kRouteTokens + wave_id_uniform()) * a.e + id;
    x_to[lane] = a.half ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
  }
}

template <int U>   // experts a lane
__global__ __launch_bounds__(64 * kRouteTokens) void moe_route_top_kernel(RouteArgs a) {
  __shared__ RouteLds<U> lds_s[kRouteTokens];
  __shared__ int id_s[kRouteTokens][32];
  __shared__ float x_s[kRouteTokens][32], top_s[kRouteTokens];
  __shared__ double total_s[kRouteTokens];
  const int lane = threadIdx.x & 63, wave = wave_id_uniform();
  const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens, t = t0 + wave;
  const int tokens = (int)min((int64_t)kRouteTokens, a.t - t0);
  if (wave < tokens) {
    float l[U], b[U];
    const size_t row = (size_t)t * a.e;
    load_row<U>(l, a.half ? (const void*)(static_cast<const uint16_t*>(a.logits) + row)
                          : (const void*)(static_cast<const float*>(a.logits) + row),
                a.half, a.whole, a.e, -__builtin_inff());
    if (a.bias)
      load_row<U>(b, a.bias, false, a.whole, a.e, 0.0f);
    else
#pragma unroll
      for (int u = 0; u < U; ++u) b[u] = 0.0f;
    float top = 0.0f;
    if (!a.sigmoid) {
      top = l[0];
#pragma unroll
      for (int u = 1; u < U; ++u) top = fmaxf(top, l[u]);
      top = wave_max(top);
      if (lane == 0) top_s[wave] = top;
      if (!a.renorm) {
        const double total = route_total(l, top);
        if (lane == 0) total_s[wave] = total;
      }
    }
    route_token<U>(a, l, b, top, lds_s[wave], id_s[wave], x_s[wave]);
  }
  __syncthreads();
  // Weights: `room` lanes a token, a pick each.
  const int room = a.k <= 8 ? 8 : a.k <= 16 ? 16 : 32;
  const int mine = threadIdx.x / room, j = threadIdx.x & (room - 1);
  if (wave * 64 >= tokens * room) return;
  const bool on = mine < tokens && j < a.k;
  const int from = on ? mine : 0, pick = on ? j : 0;
  const double x = (double)x_s[from][pick];
  double w;
  if (a.sigmoid)
    w = 1.0 / (1.0 + exp(-x));
  else
    w = route_exp((float)x, top_s[from]);
  double total = 1.0;
  if (a.renorm) {
    total = on ? w : 0.0;
    total += __shfl_xor(total, 1);
    total += __shfl_xor(total, 2);
    total += __shfl_xor(total, 4);
    if (room > 8) total += __shfl_xor(total, 8);
    if (room > 16) total += __shfl_xor(total, 16);
  } else if (!a.sigmoid) {
    total = total_s[from];
  }
  w = total == 0.0 ? 0.0 : w / total;
  if (!on) return;
  a.ids[(t0 + mine) * a.k + j] = id_s[from][pick];
  a.weights[(t0 + mine) * a.k + j] = (float)((double)a.scale * w);
}

// ---- many tokens, up to 8 picks of 256 experts ----------------------------------------
//
// Four tokens a wave, 16 lanes each, V experts a lane.  A lane keeps its best eight as
// sorted keys, so that a round of the choice is a maximum over 16 lanes and a shift in
// the lane that had it, for four tokens at once and without scalar work (a wave a token
// as above takes about 300 vector and 330 scalar instructions a token at 8 of 256
// experts, and these take turns).
//
// A key is c's step, and the expert it belongs to is looked up in the lane's c, which
// lie in LDS, when all picks are known.  Where logits of 16 bits are compared as they are,
// which are often equal, the last bits of a key are the expert's number, lower ones
// first.  Tokens whose keys do not tell, or that have a NaN, are done again in 64
// bits, by the whole wave.

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {   // of 16 lanes, in all of them
  v = max(v, dpp_u<0x128>(v));           // row_ror 8, 4, 2, 1
  v = max(v, dpp_u<0x124>(v));
  v = max(v, dpp_u<0x122>(v));
  return max(v, dpp_u<0x121>(v));
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_f<0x128>(v));
  v = fmaxf(v, dpp_f<0x124>(v));
  v = fmaxf(v, dpp_f<0x122>(v));
  return fmaxf(v, dpp_f<0x121>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<0x128>(v);
  v += dpp_f<0x124>(v);
  v += dpp_f<0x122>(v);
  return v + dpp_f<0x121>(v);
}
// k[A] and k[B] in order, the larger first.
template <int A, int B, int N>
__device__ __forceinline__ void in_order(uint32_t (&k)[N]) {
  const uint32_t a = max(k[A], k[B]), b = min(k[A], k[B]);
  k[A] = a, k[B] = b;
}
// F .. F + 3 sorted, largest first; F .. F + 7 by an odd-even merge of two of these.
template <int F, int N>
__device__ __forceinline__ void sort4(uint32_t (&k)[N]) {
  in_order<F, F + 1>(k), in_order<F + 2, F + 3>(k);
  in_order<F, F + 2>(k), in_order<F + 1, F + 3>(k);
  in_order<F + 1, F + 2>(k);
}
template <int F, int N>
__device__ __forceinline__ void sort8(uint32_t (&k)[N]) {
  sort4<F>(k), sort4<F + 4>(k);
  in_order<F, F + 4>(k), in_order<F + 1, F + 5>(k), in_order<F + 2, F + 6>(k), in_order<F + 3, F + 7>(k);
  in_order<F + 2, F + 4>(k), in_order<F + 3, F + 5>(k);
  in_order<F + 1, F + 2>(k), in_order<F + 3, F + 4>(k), in_order<F + 5, F + 6>(k);
}
// The best 8 of 16 into k[0 .. 7], sorted: of two sorted eights the larger of each place and
// its mirror, which rise and fall (or fall and rise) once, then their merge.
__device__ __forceinline__ void best8(uint32_t (&k)[16]) {
  sort8<0>(k), sort8<8>(k);
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i] = max(k[i], k[15 - i]);
  in_order<0, 4>(k), in_order<1, 5>(k), in_order<2, 6>(k), in_order<3, 7>(k);
  in_order<0, 2>(k), in_order<1, 3>(k), in_order<4, 6>(k), in_order<5, 7>(k);
  in_order<0, 1>(k), in_order<2, 3>(k), in_order<4, 5>(k), in_order<6, 7>(k);
}

// V values of a lane: 4, 8 or 16.
template <int V>
__device__ __forceinline__ void load_lane(float (&v)[V], const void* row, bool half, int e) {
  if (half) {
    const uint16_t* const p = static_cast<const uint16_t*>(row) + e;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = __uint_as_float((j & 1) ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
    }
  } else {
    const float* const p = static_cast<const float*>(row) + e;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4_t w = *reinterpret_cast<const f32x4_t*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = w[j];
    }
  }
}

template <int V>
__global__ __launch_bounds__(256) void moe_route_rows_kernel(RouteArgs a) {
  constexpr int U = V / 4;               // experts a lane where the whole wave takes a token
  constexpr int K = V < 8 ? V : 8;       // keys a lane keeps
  static_assert(V == 4 || V == 8 || V == 16, "experts a lane");
  __shared__ RouteLds<U> lds_s[4];
  __shared__ __attribute__((aligned(16))) float c_s[4][64][V + 4];   // rows 16 bytes apart at least, off the same banks
  __shared__ u32x2_t pick_s[4][4][8];
  __shared__ int fixed_s[4][4][8];
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4, wave = wave_id_uniform();
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
  if (t0 >= a.t) return;                 // waves share nothing
  const int64_t t = min(t0 + q, a.t - 1);
  const bool live = V * i < a.e;         // e is a multiple of V
  const int at = live ? V * i : 0;
  float c[V];
  const size_t row = (size_t)t * a.e;
  load_lane<V>(c, a.half ? (const void*)(static_cast<const uint16_t*>(a.logits) + row)
                         : (const void*)(static_cast<const float*>(a.logits) + row), a.half, at);
  float top = 0.0f;
  double total = 0.0;                    // of softmax scores that are not renormalized
  if (!a.sigmoid) {
    top = c[0];
#pragma unroll
    for (int u = 1; u < V; ++u) top = fmaxf(top, c[u]);
    top = row_max(live ? top : -__builtin_inff());
    if (!a.renorm) {
#pragma unroll
      for (int u = 0; u < V; ++u) total += route_exp(c[u], top);
      total = live ? total : 0.0;
      total += __shfl_xor(total, 1);
      total += __shfl_xor(total, 2);
      total += __shfl_xor(total, 4);
      total += __shfl_xor(total, 8);
    }
  }
  // c, and the bound on its error (route_token).
  const bool exact = a.bias == nullptr && (a.groups == 1 || a.best == 1);
  const bool whole_key = exact && a.half;
  float most = 1.0f;                     // the largest score, at most
  bool near = false;
#pragma unroll
  for (int u = 0; u < V; ++u) near |= c[u] != c[u];
  if (!exact) {
    constexpr float kLog2e = 1.44269504088896340736f;
    float b[V];
#pragma unroll
    for (int u = 0; u < V; ++u) b[u] = 0.0f;
    if (a.bias) load_lane<V>(b, a.bias, false, at);
    if (a.sigmoid) {
#pragma unroll
      for (int u = 0; u < V; ++u) c[u] = b[u] + __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * c[u]));
    } else {
      float sum = 0.0f;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        c[u] = c[u] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(kLog2e * (c[u] - top));
        sum += c[u];
      }
      sum = row_sum(live ? sum : 0.0f);
      most = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int u = 0; u < V; ++u) c[u] = b[u] + c[u] * most;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) near |= c[u] != c[u];   // a bias that is none
  }
  const float least = a.sigmoid ? 0x1p-21f : most * 0x1p-18f;
  auto off = [&](float v) { return exact ? 0.0f : __builtin_fmaf(fabsf(v), 0x1p-23f, least); };
  uint32_t k[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const uint32_t step = step_of(c[u]);
    k[u] = !live ? 0u : whole_key ? (step & ~0x1ffu) | (uint32_t)(511 - (at + u)) : step;
  }
  if (!whole_key)
#pragma unroll
    for (int u = 0; u < V; u += 4) *reinterpret_cast<f32x4_t*>(&c_s[wave][lane][u]) = f32x4_t{c[u], c[u + 1], c[u + 2], c[u + 3]};
  if constexpr (V == 4)
    sort4<0>(k);
  else if constexpr (V == 8)
    sort8<0>(k);
  else
    best8(k);
  const uint32_t low = whole_key ? 0x1ffu : 0u;
  // (the last bits of a negative number's step are ones)
  auto value_of = [&](uint32_t key) { return step_to((key >> 31) != 0 ? key & ~low : key | low); };

  bool open = live;                      // the lane's experts can be picked
  if (a.groups > 1) {
    const int lanes = a.lanes16;
    float c1 = value_of(k[0]), c2 = value_of(k[1]);
    best_two<1>(lanes, c1, c2);
    best_two<2>(lanes, c1, c2);
    best_two<4>(lanes, c1, c2);
    best_two<8>(lanes, c1, c2);
    const float value = a.best == 1 ? c1 : c1 + c2;
    const int own = i >> a.shift16, first = i & (lanes - 1);
    float before = 0.0f;                 // groups before this one
    // A group's lanes compare it with one other group each, in turn.
    for (int g0 = 0; g0 < a.groups; g0 += lanes) {
      const int g = g0 + first;
      const float other = __shfl(value, 16 * q + (min(g, a.groups - 1) << a.shift16));
      const bool is = g < a.groups && g != own && live;
      before += is && (other > value || (other == value && g < own)) ? 1.0f : 0.0f;
    }
    if (lanes > 1) before += other_block<1>(before);
    if (lanes > 2) before += other_block<2>(before);
    if (lanes > 4) before += other_block<4>(before);
    if (lanes > 8) before += other_block<8>(before);
    open = live && before < (float)a.top_groups;
    if (!exact) {                        // the last group that stays and the first that does not
      const float e = 1.5f * (off(c1) + off(a.best == 1 ? c1 : c2));
      const float stays = -row_max(open ? e - value : -__builtin_inff());
      const float goes = row_max(live && !open ? value + e : -__builtin_inff());
      near |= !(stays > goes);
    }
    if (!open)
#pragma unroll
      for (int j = 0; j < K; ++j) k[j] = 0u;
  }

  // A round: the largest key of the 16 lanes, and in its lane the next one.
  bool twice = false;                    // a key in two lanes
  for (int j = 0; j < a.k; ++j) {
    const uint32_t m = row_max(k[0]);
    const bool it = k[0] == m;
    twice |= __popcll(__ballot(it)) != 4;
    if (it) {
      pick_s[wave][q][j] = u32x2_t{m, (uint32_t)i};
#pragma unroll
      for (int o = 0; o + 1 < K; ++o) k[o] = k[o + 1];
      k[K - 1] = 0u;
    }
  }
  const uint32_t next = row_max(k[0]);
  wave_fence();
  const u32x2_t pick = pick_s[wave][q][i & 7];
  const bool on = i < a.k;
  const uint32_t mine = on ? pick[0] : 0u, from = on ? pick[1] & 15u : 0u;   // lane j: the j-th pick's key, and its lane
  if (V > K && !whole_key) near |= open && k[0] == 0u;   // a lane that gave all it had kept, and has more
  if (!whole_key) {                      // a pick and the one behind it, or the first that is none
    uint32_t behind = dpp_u<0x101>(mine);   // row_shl 1
    behind = i == a.k - 1 ? next : behind;
    const float v = value_of(mine), w = value_of(behind);
    near |= on && behind != 0u && !(v - w > off(v) + off(w));
  }
  int id = (int)(511u - (mine & low));
  if (!whole_key) {
    wave_fence();
    const float v = value_of(mine);
    const float* const of = c_s[wave][16 * q + from];
    int u_of = 0;
#pragma unroll
    for (int u = V - 1; u >= 0; --u) u_of = of[u] == v ? u : u_of;
    id = V * (int)from + u_of;
  }

  uint64_t again = __ballot(near);
  if (twice) again = ~(uint64_t)0;
  if (again != 0) {
    for (int r = 0; r < 4; ++r) {
      if ((again >> (16 * r) & 0xffffu) == 0 || t0 + r >= a.t) continue;   // uniform
      float l[U];
      const size_t at_r = (size_t)(t0 + r) * a.e;
      load_row<U>(l, a.half ? (const void*)(static_cast<const uint16_t*>(a.logits) + at_r)
                            : (const void*)(static_cast<const float*>(a.logits) + at_r),
                  a.half, a.whole, a.e, -__builtin_inff());
      const int id_r = route_exact(a, l, lane_of(top, 16 * r), lds_s[wave]);
      if (lane < a.k) fixed_s[wave][r][lane] = id_r;
      wave_fence();
    }
    if ((again >> (16 * q) & 0xffffu) != 0) id = fixed_s[wave][q][i & 7];
  }

  const size_t of = row + (on ? min(max(id, 0), a.e - 1) : 0);
  const float x = a.half ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[of]) : static_cast<const float*>(a.logits)[of];
  double w;
  if (a.sigmoid)
    w = 1.0 / (1.0 + exp(-(double)x));
  else
    w = route_exp(x, top);
  if (a.renorm) {
    total = on ? w : 0.0;
    total += __shfl_xor(total, 1);
    total += __shfl_xor(total, 2);
    total += __shfl_xor(total, 4);
  } else if (a.sigmoid) {
    total = 1.0;
  }
  w = total == 0.0 ? 0.0 : w / total;
  if (on && t0 + q < a.t) {
    a.ids[t * a.k + i] = id;
    a.weights[t * a.k + i] = (float)((double)a.scale * w);
  }
}

// From here on four tokens a wave are taken, from twice as many for more than 64 experts
// and four times for more than 128 (four tokens a wave against one, us in a graph.  64
// experts, softmax: 4096 tokens 3.4 against 4.8, 16385 4.6 against 10.3; 500000 of 8 64
// against 194.  128, biased: 4096 6.3 against 6.1, 8192 6.9 against 8.8, 16385 9.9 against
// 11.5, 65536 22.5 against 34.9.  256, biased: 8192 11.3 against 10.0, 16384 14.6 against
// 13.9, 24576 21.6 against 18.8, 32768 19.5 against 23.2; grouped: 8192 10.4 against 11.6,
// 16384 19.0 against 16.5, 16385 15.2 against 16.6, 24576 25.7 against 21.9, 32768 23.1
// against 27.1).  There it is about even up to 32768 tokens and goes by how many of them
// end in 64 bits, for which the other three of their wave wait.  Where the logits decide
// none does, and four tokens a wave would pay from 1024 on (256 experts: 4.2 against 4.5,
// 8192 5.3 against 8.0): the rule does not tell these apart.
constexpr int64_t kRouteRowsFrom = 4096;

hipError_t launch_moe_route(RouteArgs a, hipStream_t stream) {
  const int u = a.e <= 64 ? 1 : a.e <= 128 ? 2 : a.e <= 256 ? 4 : 8;
  auto on = [](const void* p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; };
  // The fast way takes groups of whole lanes, a power of two of them.
  const int per = a.e / a.groups, lanes = per / u;
  a.lanes = per % u == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  for (a.shift = 0; 1 << a.shift < a.lanes;) ++a.shift;
  a.whole = a.e % u == 0 && on(a.logits, a.half ? 2 * u : u < 4 ? 4 * u : 16) && on(a.bias, u < 4 ? 4 * u : 16);
  const int v = 4 * u, lanes16 = per / v;
  a.lanes16 = per % v == 0 && (lanes16 & (lanes16 - 1)) == 0 ? lanes16 : 0;
  for (a.shift16 = 0; 1 << a.shift16 < a.lanes16;) ++a.shift16;
  if (a.t >= kRouteRowsFrom * u && a.k <= 8 && u <= 4 && a.e % v == 0 && a.whole && on(a.logits, 16) && on(a.bias, 16) &&
      (a.groups == 1 || a.lanes16 > 0)) {
    const dim3 rows((uint32_t)((a.t + 15) / 16));
    if (u == 1)
      hipLaunchKernelGGL((moe_route_rows_kernel<4>), rows, dim3(256), 0, stream, a);
    else if (u == 2)
      hipLaunchKernelGGL((moe_route_rows_kernel<8>), rows, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((moe_route_rows_kernel<16>), rows, dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  const dim3 grid((uint32_t)((a.t + kRouteTokens - 1) / kRouteTokens));
  if (a.e <= 64)
    hipLaunchKernelGGL((moe_route_top_kernel<1>), grid, dim3(64 * kRouteTokens), 0, stream, a);
  else if (a.e <= 128)
    hipLaunchKernelGGL((moe_route_top_kernel<2>), grid, dim3(64 * kRouteTokens), 0, stream, a);
  else if (a.e <= 256)
    hipLaunchKernelGGL((moe_route_top_kernel<4>), grid, dim3(64 * kRouteTokens), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_route_top_kernel<8>), grid, dim3(64 * kRouteTokens), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
