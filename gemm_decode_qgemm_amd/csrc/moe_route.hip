// moe_route.hip -- the choice of experts from a router's logits (qg_moe_route).
//
//   s = softmax(l) or sigmoid(l);   c = s + bias      (the bias decides, it does not weigh)
//   experts in equal groups: a group counts the sum of its best one or two c; the
//   best groups stay;   the top k experts by c among them, ties to the lowest index;
//   w = s of the picked, over their sum where renormalized, times a scale
//
// A wave takes a token, lane l experts l, 64 + l, ...  Scores are formed in 64 bits:
// which of two experts comes first is a comparison of computed numbers, and in 32
// bits one choice in some thousands would go by rounding.  Where no bias and no sum
// of two takes part the order is that of the logits, compared as they are.
#include "layer_common.h"

namespace qg {

// A number as an unsigned one of the same order; NaN is above all, -0 is 0, none is 0.
__device__ __forceinline__ uint64_t order64(double c) {
  c += 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(c);
  if (c != c) return ~(uint64_t)0;
  return (u >> 63) != 0 ? ~u : u | (uint64_t)1 << 63;
}

__device__ __forceinline__ uint32_t wave_max32(uint32_t v) {
  auto step = [&](uint32_t o) { v = max(v, o); };
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));   // row_shr 1, 2, 4, 8
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));   // row_bcast 15, 31
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

template <int U>   // experts a lane
__global__ __launch_bounds__(256) void moe_route_top_kernel(RouteArgs a) {
  __shared__ double choice_s[4][64 * U];
  const int lane = threadIdx.x & 63, wave = wave_id_uniform();
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.t) return;              // a wave's LDS is its own
  float l[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 64 * u + lane;
    l[u] = -__builtin_inff();
    if (e < a.e)
      l[u] = a.half ? bf16_to_f32(static_cast<const uint16_t*>(a.logits)[t * a.e + e])
                    : static_cast<const float*>(a.logits)[t * a.e + e];
  }
  double s[U];
  if (a.sigmoid) {
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = 1.0 / (1.0 + exp(-(double)l[u]));
  } else {
    float top = l[0];
#pragma unroll
    for (int u = 1; u < U; ++u) top = fmaxf(top, l[u]);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    double total = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a token without a logit above -infinity has no scores; NaN stays NaN
      s[u] = l[u] == -__builtin_inff() ? 0.0 : exp((double)l[u] - (double)top);
      total += s[u];
    }
    total = wave_sum64(total);
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = total == 0.0 ? 0.0 : s[u] / total;
  }
  // Keys in the order of c.
  uint64_t key[U];
  const bool by_logit = a.bias == nullptr && (a.groups == 1 || a.best == 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 64 * u + lane;
    double c = by_logit ? (double)l[u] : s[u];
    if (a.bias && e < a.e) c += (double)a.bias[e];
    key[u] = e < a.e ? order64(c) : 0;
    if (a.groups > 1) choice_s[wave][e] = c;
  }
  if (a.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int per = a.e / a.groups;
    uint64_t mine = 0;
    if (lane < a.groups) {           // lane g: the best one or two of group g
      uint64_t k1 = 0, k2 = 0;
      double c1 = 0.0, c2 = 0.0;
      for (int i = 0; i < per; ++i) {
        const double c = choice_s[wave][lane * per + i];
        const uint64_t k = order64(c);
        if (k > k1) {
          k2 = k1, c2 = c1;
          k1 = k, c1 = c;
        } else if (k > k2) {
          k2 = k, c2 = c;
        }
      }
      mine = a.best == 1 ? k1 : order64(c1 + c2);
    }
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t other = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), g) << 32 |
                             (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
      before += other > mine || (other == mine && g < lane);
    }
    const uint64_t open = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((open >> ((64 * u + lane) / per & 63) & 1) == 0) key[u] = 0;
  }
  // k rounds: the largest key of the wave, then the lowest expert that has it.
  double w = 0.0;                    // lane j: the j-th pick's score
  int id = 0;
  for (int j = 0; j < a.k; ++j) {
    uint64_t m = key[0];
#pragma unroll
    for (int u = 1; u < U; ++u) m = max(m, key[u]);
    const uint32_t hi = wave_max32((uint32_t)(m >> 32));
    const uint32_t lo = wave_max32((uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u);
    m = (uint64_t)hi << 32 | lo;
    bool found = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (found) continue;           // uniform
      const uint64_t has = __ballot(key[u] == m);
      if (has == 0) continue;
      found = true;
      const int at = __builtin_ctzll(has);
      if (lane == at) key[u] = 0;
      const double v = __shfl(s[u], at);
      if (lane == j) w = v, id = 64 * u + at;
    }
  }
  if (a.renorm) {
    const double total = wave_sum64(w);
    w = total == 0.0 ? 0.0 : w / total;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = id;
    a.weights[t * a.k + lane] = (float)((double)a.scale * w);
  }
}

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)((a.t + 3) / 4));
  if (a.e <= 64)
    hipLaunchKernelGGL((moe_route_top_kernel<1>), grid, dim3(256), 0, stream, a);
  else if (a.e <= 128)
    hipLaunchKernelGGL((moe_route_top_kernel<2>), grid, dim3(256), 0, stream, a);
  else if (a.e <= 256)
    hipLaunchKernelGGL((moe_route_top_kernel<4>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_route_top_kernel<8>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
