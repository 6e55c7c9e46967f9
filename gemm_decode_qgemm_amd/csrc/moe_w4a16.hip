// moe_w4a16.hip -- a whole mixture-of-experts layer for up to 64 tokens on
// packed INT4 group-32 experts (qg_moe_w4a16).
//
//   l = x Wr^T;  the top k experts of a token (ties: the lowest index);
//   p = softmax over the picked logits, or over all of them;
//   y = sum over the picked e of p_e W2_e (silu(Wg_e x) * (Wu_e x))
// with the products of qgemm_w4a16: exact bf16 (128 + q) times bf16
// activations, fp32 sums, the group scale and -(128 + zp) times the group sum
// of x applied per group in fp32.  The hidden activation is rounded to bf16
// once, as the second product's operand (up to 4 tokens it is the sum of two bf16,
// which costs nothing there); all else is fp32.
//
// Launches, with no atomics between workgroups (bit-identical repeats):
//   router      logits in fp32
//   route       the tokens of every expert; up to 8 tokens the next launch
//               finds them itself while its workgroups all run at once
//   gate and up the two products of a few hidden columns of one expert, and
//               silu(g) u of its tokens
//   down        up to 4 tokens: the weighted sum over a token's picks; above: fp32
//               results per (token, pick)
//   combine     above 4 tokens: the weighted sum, in order of rank
// The rank of expert e for a token is the number of experts before it, so "which
// tokens picked e" takes one ballot per 64 experts and token (route), and a token's
// pick number is that rank.  A workgroup that ranks by itself takes the largest
// logit left, once per pick; for one token it compares all of them at once in LDS,
// with 16 waves (1 token, 8 of 128 experts of 768 x 2048: 15.9 us against 17.5).
//
// Two forms of the product:
//  * one to 4 tokens of an expert: the 4x4x4 sixteen-block matrix instruction
//    with lane = weight row (the mapping of gemv_w4a16_mx4.hip), K split over
//    waves and summed in LDS;
//  * more: 16x16x32 with the tokens staged in LDS, one wave per 16 weight rows
//    through all of K (the mapping of the LDS form of gemm_w4a16_mfma.hip),
//    MT = 1 or 2 tiles of 16 tokens at a time.
//
// The least a call can do is read the weights of the experts that were picked, 37/64
// byte each.  Measured, whole layer: 1 token, 8 of 128 experts of 768 x 2048, 15.9 us
// (three launches that wait for each other; 3.4 us of bytes); 1 token, 2 of 8 of
// 14336 x 4096, 46 us (4.4 TB/s); 17 tokens, 6 of 64 of 1024 x 2048, 46 to 56 us (10 us
// of it the small launches, the rest short columns of K); 64 tokens, 2 of 8 of
// 14336 x 4096, 214 to 232 us (3.5 to 3.8 TB/s): there the vector instructions that unpack
// codes (62 % of a SIMD's issue without the matrix ones) and the matrix pipe (34 %)
// take turns; exactly 16 tokens an expert, one tile, take 195 us, 22 to 32 take 260.
#include <type_traits>

#include "layer_common.h"
#include "w4_common.h"

namespace qg {

constexpr int kFewTokens = 4;         // up to these, the down launch adds a token's picks itself

struct MoeArgs {
  const uint16_t *x, *router;
  const uint8_t *gate_up, *down;
  size_t gate_up_bytes, down_bytes;   // per expert
  int t, h, e, inter, k, renorm;
  int direct;                         // units of the expert launches: experts, with tokens or not
  int own;                            // gate and up ranks the logits itself: no lists
  float* logits;                      // [t, e]
  float* picked;                      // [t * k] logits in order of rank
  int32_t* count;                     // [e] tokens of an expert
  int32_t* list;                      // [e][64] their picks, t k + rank
  int32_t* expert_of;                 // [t * k] experts in order of rank
  uint16_t* hidden;                   // [t * k, inter]; up to 4 tokens: [2][t * k, inter], a sum of two
  float* part;                        // [t * k, h]
  void* y;
  int y_f32;
};

// ---- router ---------------------------------------------------------------

// A workgroup per expert and 4 tokens, summed over its lanes in a fixed order.
__global__ __launch_bounds__(256) void moe_router_gemv_kernel(MoeArgs a) {
  __shared__ float red[4][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int e = blockIdx.x, t0 = 4 * blockIdx.y;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = tid * 8; c < a.h; c += 2048) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(a.router + (size_t)e * a.h + c);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(a.x + (size_t)min(t0 + m, a.t - 1) * a.h + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[m] = __builtin_fmaf(__uint_as_float(x[i] << 16), __uint_as_float(w[i] << 16), acc[m]);
        acc[m] = __builtin_fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(w[i] & 0xffff0000u), acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) acc[m] += __shfl_xor(acc[m], o);
    if (lane == 0) red[wave][m] = acc[m];
  }
  __syncthreads();
  if (tid < 4 && t0 + tid < a.t) a.logits[(size_t)(t0 + tid) * a.e + e] = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
}

// 16 experts x 16 tokens per workgroup, its 16 waves taking 32 k in turn.
__global__ __launch_bounds__(1024) void moe_router_mfma_kernel(MoeArgs a) {
  __shared__ f32x4_t red[16][64];
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = wave_id_uniform();
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const uint16_t* const w = a.router + (size_t)min(e0 + i, a.e - 1) * a.h + 8 * q;
  const uint16_t* const x = a.x + (size_t)min(t0 + i, a.t - 1) * a.h + 8 * q;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = wave * 32; c < a.h; c += 2048) {      // four steps' loads in flight together
    u32x4_t xv[4], wv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      xv[u] = wv[u] = u32x4_t{0u, 0u, 0u, 0u};
      if (c + 512 * u < a.h) {
        xv[u] = *reinterpret_cast<const u32x4_t*>(x + c + 512 * u);
        wv[u] = *reinterpret_cast<const u32x4_t*>(w + c + 512 * u);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[u]), __builtin_bit_cast(bf16x8_t, wv[u]),
                                                    acc, 0, 0, 0);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  f32x4_t v = red[0][lane];
  for (int u = 1; u < 16; ++u) {
    const f32x4_t r = red[u][lane];
    v = f32x4_t{v[0] + r[0], v[1] + r[1], v[2] + r[2], v[3] + r[3]};
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = t0 + 4 * q + j;
    if (t < a.t && e0 + i < a.e) a.logits[(size_t)t * a.e + e0 + i] = v[j];
  }
}

// ---- routing -------------------------------------------------------------------

// The largest of the wave's 64 values.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](uint32_t o) { v = max(v, o); };
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));   // row_shr 1, 2, 4, 8
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));   // row_bcast 15, 31
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A logit as an unsigned number of the same order; NaN is above all, -0 is 0.
__device__ __forceinline__ uint32_t order_key(float l) {
  l += 0.0f;
  const uint32_t u = __float_as_uint(l);
  if (l != l) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One token: the expert of rank `want`.  Workgroups of 1024 threads.
struct MoePlan {
  uint32_t key[512];
  int count[512];
  int expert;
};

__device__ int moe_plan(const MoeArgs& a, int want, MoePlan& p) {
  const int tid = threadIdx.x;
  if (tid < a.e) p.key[tid] = order_key(a.logits[tid]);
  if (tid < 512) p.count[tid] = 0;
  __syncthreads();
  int width = 64;                    // lanes for the experts, 1024 / width parts of the comparison
  while (width < a.e) width *= 2;
  const int parts = 1024 / width, e = tid & (width - 1), part = tid / width;
  if (e < a.e) {
    const uint32_t mine = p.key[e];
    int c = 0;
#pragma unroll 8
    for (int o = a.e * part / parts; o < a.e * (part + 1) / parts; ++o) {
      const uint32_t u = p.key[o];
      c += u > mine || (u == mine && o < e);
    }
    atomicAdd(&p.count[e], c);       // integers in LDS: no order to depend on
  }
  __syncthreads();
  if (tid < a.e && p.count[tid] == want) p.expert = tid;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(p.expert);
}

// The first `upto` experts of token t in order of rank, by a wave: take(rank,
// expert).  A round is the largest key of the wave, then the lowest expert that
// has it (about 50 ns).
template <class Take>
__device__ __forceinline__ void moe_top(const MoeArgs& a, int t, int upto, Take take) {
  const int lane = threadIdx.x & 63;
  uint32_t key[8];                   // of expert 64 u + lane; no logit's key is 0
#pragma unroll
  for (int u = 0; u < 8; ++u) key[u] = 64 * u + lane < a.e ? order_key(a.logits[(size_t)t * a.e + 64 * u + lane]) : 0u;
  for (int j = 0; j < upto; ++j) {
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = max(m, key[u]);
    m = wave_max(m);
    int at = -1;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (64 * u >= a.e || at >= 0) continue;    // uniform
      const uint64_t has = __ballot(key[u] == m);
      if (has == 0) continue;
      const int l = __builtin_ctzll(has);
      at = 64 * u + l;
      if (lane == l) key[u] = 0u;
    }
    take(j, at);
  }
}

// Above one token, unless the gate and up launch does it: a workgroup per expert
// ranks it for every token.
__global__ __launch_bounds__(512) void moe_route_kernel(MoeArgs a) {
  __shared__ int rank[64];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int expert = blockIdx.x;
  // wave w: tokens w, w + 8, ..., all their loads of 64 experts in flight together
  uint32_t mine[8];
  int c[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int t = wave + 8 * u;
    mine[u] = t < a.t ? order_key(a.logits[(size_t)t * a.e + expert]) : 0u;
    c[u] = 0;
  }
  for (int o0 = 0; o0 < a.e; o0 += 64) {
    const int o = o0 + lane;
    uint32_t key[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = wave + 8 * u;
      key[u] = t < a.t && o < a.e ? order_key(a.logits[(size_t)t * a.e + o]) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      c[u] += __popcll(__ballot(o < a.e && (key[u] > mine[u] || (key[u] == mine[u] && o < expert))));
  }
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (lane == 0 && wave + 8 * u < a.t) rank[wave + 8 * u] = c[u];
  __syncthreads();
  if (wave != 0) return;
  const bool sel = lane < a.t && rank[lane < a.t ? lane : 0] < a.k;
  const uint64_t mask = __ballot(sel);
  if (lane == 0) a.count[expert] = __popcll(mask);
  if (sel) {
    const int slot = lane * a.k + rank[lane];
    a.list[expert * 64 + __popcll(mask & (((uint64_t)1 << lane) - 1))] = slot;
    a.picked[slot] = a.logits[(size_t)lane * a.e + expert];
    a.expert_of[slot] = expert;
  }
}

// The expert of a unit after the route launch: the unit-th that has tokens, or -1.
__device__ __forceinline__ int moe_active(const MoeArgs& a, int unit, int& n) {
  const int lane = threadIdx.x & 63;
  int cnt[8], expert = -1, seen = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) cnt[u] = 64 * u + lane < a.e ? a.count[64 * u + lane] : 0;
  n = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint64_t mask = __ballot(cnt[u] > 0);
    const bool me = cnt[u] > 0 && __popcll(mask & (((uint64_t)1 << lane) - 1)) == unit - seen;
    const uint64_t hit = __ballot(me);
    if (hit != 0) {
      const int at = __builtin_ctzll(hit);
      expert = 64 * u + at;
      n = __builtin_amdgcn_readlane(cnt[u], at);
    }
    seen += __popcll(mask);
  }
  return expert;
}

// Where the workgroups of the gate and up launch rank the logits themselves: of[u]
// is the expert of slot 64 u + lane (t k + rank).  The expert of a unit and its
// picks (lane m: the m-th, the last one past it), or -1: units are experts
// (direct), or slots, of which the first with its expert works for all.
constexpr int kOwnTokens = 8;
constexpr int kOwnSlots = kOwnTokens * 32 / 64;

__device__ __forceinline__ int moe_own(const MoeArgs& a, const int (&of)[kOwnSlots], int unit, int* list, int& n,
                                       int& pick) {
  const int lane = threadIdx.x & 63;
  int expert = unit;
  if (!a.direct) {
#pragma unroll
    for (int u = 0; u < kOwnSlots; ++u)
      if (unit >> 6 == u) expert = __builtin_amdgcn_readlane(of[u], unit & 63);
  }
  n = 0;
  int first = -1;
#pragma unroll
  for (int u = 0; u < kOwnSlots; ++u) {
    const bool mine = of[u] == expert;
    const uint64_t mask = __ballot(mine);
    if (mask == 0) continue;
    if (first < 0) first = 64 * u + __builtin_ctzll(mask);
    if (mine) list[n + __popcll(mask & (((uint64_t)1 << lane) - 1))] = 64 * u + lane;
    n += __popcll(mask);
  }
  if (n == 0 || (!a.direct && first != unit)) return -1;
  // wave-private: a wave's LDS operations complete in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  pick = list[min(lane, n - 1)];
  return expert;
}

// ---- the experts' products -----------------------------------------------------

constexpr int kMoeXRow = 288;     // LDS bytes of a token's 128 k (two runs of 128, 16 apart)
constexpr int kMoeXPair = 144;

struct MoeSlot {                  // of one wave
  uint8_t x[4 * kMoeXRow];
  float sum[4][4];                // group sums of x: [group][token]
};

// A half tile (128 k) of a wave's 32 weight rows and the activations it meets.
struct MoeHalf {
  const uint8_t* tile;
  int half;
  const uint16_t* x;              // this lane's activation row, its first k
};

// acc[m] += dequant(W)[row] . x_m over the wave's units u0, u0 + step, ...
// below `units`, for M rows of activations (lanes copy 4); at(u) names unit u.  Lane l
// holds row l & 31 of the half block `hb` and the group pair l >> 5, and copies
// 8 k of activation row l >> 4.
template <int M, bool PF, class At>
__device__ __forceinline__ void moe_mx4(float (&acc)[M], int hb, int u0, int units, int step, MoeSlot& slot, At at) {
  using L = W4Layout<false>;
  const int lane = threadIdx.x & 63, lg = lane >> 5, sm = lane >> 4, sc = lane & 15;
  const int row = 32 * hb + (lane & 31);
  const int swr = sm * kMoeXRow + 16 * sc + (sc >= 8 ? 16 : 0);
  const int srd = (lane & 3) * kMoeXRow + lg * kMoeXPair;
  const uint32_t mask_s = __builtin_amdgcn_readfirstlane(0x000F000Fu);
  uint32_t magic_v = 0x43004300u;
  asm volatile("" : "+v"(magic_v));
  uint32_t ones_v = 0x3f803f80u;
  asm volatile("" : "+v"(ones_v));
  auto load = [&](Half32Regs& r, u32x4_t& xv, int u) {
    const MoeHalf h = at(u);
    L::load(r, h.tile, h.half, lg, row);
    xv = *reinterpret_cast<const u32x4_t*>(h.x + 8 * sc);
  };
  auto compute = [&](const Half32Regs& r, const u32x4_t& xv) {
    float xp = dot2_bf16(xv.x, ones_v, 0.0f);
    xp = dot2_bf16(xv.y, ones_v, xp);
    xp = dot2_bf16(xv.z, ones_v, xp);
    xp = dot2_bf16(xv.w, ones_v, xp);
    xp += dpp_mov<0xB1>(xp);
    xp += dpp_mov<0x4E>(xp);
    // wave-private slot: a wave's LDS operations complete in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    *reinterpret_cast<u32x4_t*>(slot.x + swr) = xv;
    if ((sc & 3) == 0) slot.sum[sc >> 2][sm] = xp;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      u32x4_t xa[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) xa[q] = *reinterpret_cast<const u32x4_t*>(slot.x + srd + 64 * jj + 16 * q);
      f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const u32x2_t b = {code_pair(r.c[jj][t >> 1], 2 * (t & 1), mask_s, magic_v),
                           code_pair(r.c[jj][t >> 1], 2 * (t & 1) + 1, mask_s, magic_v)};
        const u32x4_t xq = xa[t >> 1];
        d = mfma_4x4x4((t & 1) ? u32x2_t{xq.z, xq.w} : u32x2_t{xq.x, xq.y}, b, d);
      }
      const float s = L::scale(r.sc, jj, 1.0f);
      const f32x4_t xg = *reinterpret_cast<const f32x4_t*>(&slot.sum[2 * lg + jj][0]);
      const float zb = (float)(L::zero(r, jj) | 0x80u);
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = __builtin_fmaf(s, __builtin_fmaf(-zb, xg[m], d[m]), acc[m]);
    }
  };
  if constexpr (!PF) {
    for (int u = u0; u < units; u += step) {
      Half32Regs r;
      u32x4_t xv;
      load(r, xv, u);
      compute(r, xv);
    }
    return;
  }
  // PF: two register sets in turn, the next unit's loads in flight while this
  // one computes
  int u = u0;
  if (u >= units) return;
  Half32Regs ra, rb;
  u32x4_t xa, xb;
  load(ra, xa, u);
  __builtin_amdgcn_sched_barrier(0);
  while (true) {
    if (u + step >= units) { compute(ra, xa); break; }
    load(rb, xb, u + step);
    __builtin_amdgcn_sched_barrier(0);
    compute(ra, xa);
    u += step;
    if (u + step >= units) { compute(rb, xb); break; }
    load(ra, xa, u + step);
    __builtin_amdgcn_sched_barrier(0);
    compute(rb, xb);
    u += step;
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g)) * u;
}

// A hidden value as a sum of two bf16, for the down launch of a few tokens: its
// matrix instruction has four rows for one token.
__device__ __forceinline__ void store_hidden2(const MoeArgs& a, size_t at, float f) {
  const uint32_t hi = f32_to_bf16_rne(f);
  a.hidden[at] = (uint16_t)hi;
  a.hidden[(size_t)a.t * a.k * a.inter + at] = (uint16_t)f32_to_bf16_rne(f - bf16_to_f32(hi));
}

// One token.  A workgroup of 16 waves owns the gate and up rows of 32 hidden
// columns of one pick, 8 waves each, K split over them.  Two workgroups per CU
// (64 VGPRs) rather than a second register set.
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(8))) void moe_gate_up_one_kernel(MoeArgs a) {
  union Shared {
    MoePlan plan;
    MoeSlot slot[16];
    float red[16][64];
  };
  __shared__ __attribute__((aligned(16))) Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int blk = wave >> 3, kw = wave & 7;
  const int tile = blockIdx.x, pick = blockIdx.y;
  const int expert = moe_plan(a, pick, sh.plan);
  if (tile == 0 && tid == 0) {
    a.expert_of[pick] = expert;
    a.picked[pick] = a.logits[expert];
  }
  __syncthreads();                   // the plan's LDS becomes the waves' slots
  const int rb = (tile >> 1) + blk * (a.inter >> 6);
  const uint8_t* const tiles = a.gate_up + expert * a.gate_up_bytes + (size_t)rb * (a.h >> 8) * kTileBytes;
  float acc[1] = {0.0f};
  moe_mx4<1, false>(acc, tile & 1, kw, a.h >> 7, 8, sh.slot[wave], [&](int u) {
    return MoeHalf{tiles + (size_t)(u >> 1) * kTileBytes, u & 1, a.x + (size_t)u * 128};
  });
  __syncthreads();
  sh.red[wave][lane] = acc[0];
  __syncthreads();
  if (tid >= 32) return;
  float v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < 16; ++w) v[w >> 3] += sh.red[w][tid] + sh.red[w][tid + 32];
  store_hidden2(a, (size_t)pick * a.inter + 32 * tile + tid, silu_mul(v[0], v[1]));
}

// The softmax denominator of a token's picks, relative to its first logit.
__device__ __forceinline__ float moe_total(const MoeArgs& a, int t, const float* l) {
  float total = 0.0f;
  if (a.renorm) {
    for (int j = 0; j < a.k; ++j) total += expf(l[j] - l[0]);
  } else {
    for (int e = threadIdx.x & 63; e < a.e; e += 64) total += expf(a.logits[(size_t)t * a.e + e] - l[0]);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
  }
  return total;
}

// Up to 4 tokens: 16 rows of a token's output through all its picks, 16 waves
// taking 256-k tiles of the picks in turn, the picks' weights applied with the
// group scales, so that neither results per pick nor a combining launch are
// needed.  Lane (i, a) holds row i of the 16 and groups a and 4 + a of the tile:
// half the rows of the mapping above and twice the workgroups (2 picks of 14336 x
// 4096: 14 us against 21 with 32 rows and 128 workgroups).  Tokens that share
// an expert read it once each, from L2 the second time (a row block's
// workgroups of all tokens go to the same XCD where h / 16 is a multiple of 8).
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(8))) void moe_down_few_kernel(MoeArgs a) {
  struct Slot {                      // of one wave: both parts of the hidden values of a tile
    uint8_t x[2][512 + 16];          // (16 bytes apart: the operand reads of lanes 4j and 4j + 1 on other banks)
    float sum[2][8];                 // their group sums
  };
  __shared__ __attribute__((aligned(16))) Slot slots[16];
  __shared__ float red[16][64];
  __shared__ float p[32];
  __shared__ int expert[32];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int i = lane & 15, q = lane >> 4, c = lane & 31, part = lane >> 5;
  const int row = 16 * (blockIdx.x & 3) + i;             // of the 64-row block
  const int token = blockIdx.y;
  const float* const picked = a.picked + token * a.k;
  const float total = moe_total(a, token, picked);
  if (tid < a.k) {
    p[tid] = expf(picked[tid] - picked[0]) / total;
    expert[tid] = a.expert_of[token * a.k + tid];
  }
  __syncthreads();
  const int kt_count = a.inter >> 8;
  const size_t block = (size_t)(blockIdx.x >> 2) * kt_count * kTileBytes;
  const uint16_t* const hidden = a.hidden + (size_t)(part * a.t + token) * a.k * a.inter + 8 * c;
  const uint32_t mask_s = __builtin_amdgcn_readfirstlane(0x000F000Fu);
  uint32_t magic_v = 0x43004300u;
  asm volatile("" : "+v"(magic_v));
  uint32_t ones_v = 0x3f803f80u;
  asm volatile("" : "+v"(ones_v));
  Slot& slot = slots[wave];
  float acc = 0.0f;
  for (int u = wave; u < a.k * kt_count; u += 16) {
    const int j = __builtin_amdgcn_readfirstlane(u / kt_count), kt = u - j * kt_count;
    const BufView v(a.down + __builtin_amdgcn_readfirstlane(expert[j]) * a.down_bytes + block + (size_t)kt * kTileBytes,
                    kTileBytes);
    u32x4_t w[2];
    uint32_t sc[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      w[g] = v.b128<true>((uint32_t)((4 * g + q) * kTileRows + row) * 16u);
      sc[g] = v.b16((uint32_t)(kScaleOff + row * 16 + 8 * g + 2 * q));
    }
    const uint32_t zw = v.b32((uint32_t)(kZeroOff + row * 4));
    const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(hidden + (size_t)j * a.inter + (size_t)kt * 256);
    float xp = dot2_bf16(xv.x, ones_v, 0.0f);
    xp = dot2_bf16(xv.y, ones_v, xp);
    xp = dot2_bf16(xv.z, ones_v, xp);
    xp = dot2_bf16(xv.w, ones_v, xp);
    xp += dpp_mov<0xB1>(xp);
    xp += dpp_mov<0x4E>(xp);
    // wave-private slot: a wave's LDS operations complete in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    *reinterpret_cast<u32x4_t*>(slot.x[part] + 16 * c) = xv;
    if ((c & 3) == 0) slot.sum[part][c >> 2] = xp;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const u32x2_t xa = *reinterpret_cast<const u32x2_t*>(slot.x[lane & 1] + 64 * (4 * g + q) + 8 * t);
        const u32x2_t b = {code_pair(w[g][t >> 1], 2 * (t & 1), mask_s, magic_v),
                           code_pair(w[g][t >> 1], 2 * (t & 1) + 1, mask_s, magic_v)};
        d = mfma_4x4x4(xa, b, d);
      }
      const float zb = (float)((zw >> (16 * g + 4 * q) & 15u) | 0x80u);
      const float x = slot.sum[0][4 * g + q] + slot.sum[1][4 * g + q];
      acc = __builtin_fmaf(p[j] * fp16_to_f32(sc[g]), __builtin_fmaf(-zb, x, d[0] + d[1]), acc);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (tid >= 16) return;
  float y = 0.0f;
#pragma unroll
  for (int u = 0; u < 16; ++u) y += (red[u][tid] + red[u][tid + 16]) + (red[u][tid + 32] + red[u][tid + 48]);
  const size_t at = (size_t)token * a.h + 16 * blockIdx.x + tid;
  if (a.y_f32)
    static_cast<float*>(a.y)[at] = y;
  else
    static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_bf16_rne(y);
}

// A barrier for LDS alone: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct MoeTile {                  // one 256-k tile of a wave's 16 rows: lane (i, a)
  u32x4_t c0, c1;                 // chunks of groups a and 4 + a, row 16t + i
  u32x4_t sc;                     // the row's 8 scales
  uint32_t zw;                    // and zero points
};

// acc[mt][e] += row 16t + i of the block times activation row 16 mt + 4a + e,
// over the tiles kt0 .. kt0 + count - 1 of K.  TH threads (`tid` among them)
// copy the 16 MT activation rows of a 256-k tile into one of two LDS buffers:
// 16-byte piece c of row r at 32 r + (c ^ (r & 15)), so that the operand reads of
// 16 lanes, one row each, fall on distinct banks; xr: this thread's rows
// tid / 32 + (TH / 32) j.  Codes go two tiles ahead, activations one (through
// registers).  The workgroup's waves pass `steps` >= count barriers together.
//
// Each group is as short as it goes: the zero point is taken off four codes at
// a time, as whole bytes 16 + q - zp; one byte permute each then gives the bf16
// pairs 144 + (q - zp), exactly; a product of x with -144 in every slot (a
// constant operand) takes the 144 off again, so that one multiply-add per output
// is left.  -(128 + zp) as the second operand instead took 26 vector
// instructions a group where this takes 18, and -144 X through LDS as the
// first value of the accumulator made LDS the bound at 32 rows.
template <int MT, int TH>
__device__ __forceinline__ void moe_mx16(f32x4_t (&acc)[MT], const uint8_t* tiles, int t, int kt0, int count, int steps,
                                         const uint16_t* (&xr)[MT * 512 / TH], int tid, uint8_t* xs) {
  constexpr int NP = MT * 512 / TH;
  const int lane = tid & 63, i = lane & 15, a = lane >> 4;
  uint32_t m144 = 0xc310c310u;     // bf16 pair (-144, -144), kept in registers
  asm volatile("" : "+v"(m144));
  const u32x4_t minus4 = {m144, m144, m144, m144};
  const bf16x8_t minus = __builtin_bit_cast(bf16x8_t, minus4);
  const f32x4_t zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  const int pc = tid & 31, pr = tid >> 5;
  auto load_w = [&](MoeTile& w, int kt) {
    const BufView v(tiles + (size_t)kt * kTileBytes, kTileBytes);
    const uint32_t row = (uint32_t)(16 * t + i), r0 = (uint32_t)a * kTileRows + row;
    w.c0 = v.b128<true>(r0 * 16u);
    w.c1 = v.b128<true>((r0 + 4 * kTileRows) * 16u);
    w.sc = v.b128<false>(kScaleOff + row * 16u);
    w.zw = v.b32(kZeroOff + row * 4u);
  };
  auto load_x = [&](u32x4_t (&x)[NP], int kt) {
#pragma unroll
    for (int j = 0; j < NP; ++j) x[j] = *reinterpret_cast<const u32x4_t*>(xr[j] + (size_t)kt * 256 + 8 * pc);
  };
  auto store_x = [&](const u32x4_t (&x)[NP], int buf) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int r = pr + TH / 32 * j;
      *reinterpret_cast<u32x4_t*>(xs + buf * (MT * 8192) + 16 * (32 * r + (pc ^ (r & 15)))) = x[j];
    }
  };
  auto compute = [&](MoeTile& w, int buf) {
    transpose_rows4(w.c0);
    transpose_rows4(w.c1);
    const uint8_t* const xb = xs + buf * (MT * 8192);
    // bytes 16 - zp of groups 0, 2, 4, 6 and 1, 3, 5, 7
    const uint32_t z0 = 0x10101010u - (w.zw & 0x0F0F0F0Fu), z1 = 0x10101010u - ((w.zw >> 4) & 0x0F0F0F0Fu);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const uint32_t dw = g < 4 ? w.c0[g] : w.c1[g - 4];
      const uint32_t z = __builtin_amdgcn_perm(0u, (g & 1) ? z1 : z0, 0x01010101u * (uint32_t)(g >> 1));
      const uint32_t lo = (dw & 0x0F0F0F0Fu) + z, hi = ((dw >> 4) & 0x0F0F0F0Fu) + z;   // bytes 16 + q - zp
      const u32x4_t bp = {__builtin_amdgcn_perm(0x43434343u, lo, 0x04020400u),
                          __builtin_amdgcn_perm(0x43434343u, hi, 0x04020400u),
                          __builtin_amdgcn_perm(0x43434343u, lo, 0x04030401u),
                          __builtin_amdgcn_perm(0x43434343u, hi, 0x04030401u)};
      const float s = fp16_to_f32((w.sc[g >> 1] >> (16 * (g & 1))) & 0xffffu);
      bf16x8_t av[MT];
      f32x4_t d[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(xb + 16 * (32 * (16 * mt + i) + ((4 * g + a) ^ i)));
        av[mt] = __builtin_bit_cast(bf16x8_t, x);
        d[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[mt], minus, zero4, 0, 0, 0);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        d[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[mt], __builtin_bit_cast(bf16x8_t, bp), d[mt], 0, 0, 0);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] = __builtin_fmaf(s, d[mt][e], acc[mt][e]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  MoeTile w0, w1, w2;
  u32x4_t x[NP];
  const int last = kt0 + max(count, 1) - 1;    // (no tile: the first one is read and not used)
  load_x(x, kt0);
  load_w(w0, kt0);
  store_x(x, 0);
  load_w(w1, min(kt0 + 1, last));
  load_x(x, min(kt0 + 1, last));
  lds_barrier();
  // Tile kt0 + k in LDS buffer k & 1 and set k % 3; the loads past the end
  // read the last tile again and are not used.
  auto step = [&](int k, MoeTile& now, MoeTile& later) {
    load_w(later, min(kt0 + k + 2, last));
    __builtin_amdgcn_sched_barrier(0);
    store_x(x, (k + 1) & 1);
    load_x(x, min(kt0 + k + 2, last));
    __builtin_amdgcn_sched_barrier(0);
    if (k < count) compute(now, k & 1);        // uniform
    lds_barrier();
  };
  for (int k = 0;;) {
    step(k, w0, w2);
    if (++k >= steps) break;
    step(k, w1, w0);
    if (++k >= steps) break;
    step(k, w2, w1);
    if (++k >= steps) break;
  }
}

// Above one token, 8 waves.  kGateUp: a workgroup owns the gate and up rows of
// 64 hidden columns, four waves each.  kDownWide: two neighbouring 64-row blocks
// of the down matrix, four waves each.  kDownDeep: one block, four waves on each
// half of K: twice the workgroups with half the work each, for grids that
// would leave CUs idle otherwise.  kGateUpFew (32 hidden columns) and kDownFew (one
// block): the matrix instruction of four tokens alone, an expert's tokens four at
// a time with its weight read again (from L2) for each four, without LDS tiles or a
// second register set, so that four workgroups fit a CU instead of two.
enum MoeForm { kGateUp, kGateUpFew, kDownWide, kDownDeep, kDownFew };

template <bool DEEP>
union MoeShared {
  MoeSlot slot[8];
  float red[8][4][64];
  uint8_t x[2][(DEEP ? 4 : 2) * 8192];       // deep: a half of K each; else one piece
  f32x4_t other[4][2][64];                   // results of the waves 4 .. 7
};
union MoeSharedFew {
  MoeSlot slot[8];
  float red[8][4][64];
};

constexpr bool is_few(MoeForm f) { return f == kGateUpFew || f == kDownFew; }

template <MoeForm F>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(is_few(F) ? 8 : 4))) void moe_expert_kernel(
    MoeArgs a) {
  constexpr bool FEW = is_few(F), UP = F == kGateUp || F == kGateUpFew, DOWN = !UP;
  constexpr bool DEEP = F == kDownDeep || F == kDownFew;
  __shared__ __attribute__((aligned(16))) std::conditional_t<FEW, MoeSharedFew, MoeShared<DEEP>> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform(), tile = blockIdx.x;
  __shared__ int slots[kOwnSlots * 64], lists[8][kOwnTokens];
  int n, expert, pick;                       // lane m of pick: the expert's m-th pick
  if (a.own) {
    const int count = a.t * a.k;
    if constexpr (UP) {
      if (wave < a.t) {
        const bool tell = tile == 0 && blockIdx.y == 0;
        moe_top(a, wave, a.k, [&](int j, int at) {
          if (lane != 0) return;
          slots[wave * a.k + j] = at;
          if (!tell) return;
          a.expert_of[wave * a.k + j] = at;
          a.picked[wave * a.k + j] = a.logits[(size_t)wave * a.e + at];
        });
      }
      __syncthreads();
    }
    int of[kOwnSlots];
#pragma unroll
    for (int u = 0; u < kOwnSlots; ++u)
      of[u] = 64 * u + lane >= count ? -1 : UP ? slots[64 * u + lane] : a.expert_of[64 * u + lane];
    expert = moe_own(a, of, blockIdx.y, lists[wave], n, pick);
    if (expert < 0) return;                  // uniform over the workgroup
  } else if (a.direct) {
    expert = blockIdx.y;
    pick = a.list[expert * 64 + lane];
    n = ((const __attribute__((address_space(4))) int*)a.count)[expert];
    if (n == 0) return;
  } else {
    expert = moe_active(a, blockIdx.y, n);
    if (expert < 0) return;
    pick = a.list[expert * 64 + min(lane, n - 1)];
  }
  const int blk = wave >> 2;
  const int kdim = DOWN ? a.inter : a.h, kt_count = kdim >> 8;
  const int rb = UP ? (FEW ? tile >> 1 : tile) + blk * (a.inter >> 6) : DEEP ? tile : 2 * tile + blk;
  const uint8_t* const tiles = (DOWN ? a.down + expert * a.down_bytes : a.gate_up + expert * a.gate_up_bytes) +
                               (size_t)rb * kt_count * kTileBytes;
  auto source = [&](int m) {                 // activation row of the m-th pick (the last one past it)
    const int s = __shfl(pick, m < n ? m : n - 1);
    return DOWN ? a.hidden + (size_t)s * a.inter : a.x + (size_t)(s / a.k) * a.h;
  };

  if (FEW || n <= 4) {
    // (block, 32-row half, one of 2 parts of K), or (half, one of 4) in the deep
    // forms of down, (block, one of 4) in the few form of gate and up
    constexpr bool HALF = F == kGateUpFew;
    constexpr int KP = DEEP || HALF ? 4 : 2;
    const int hb = HALF ? tile & 1 : DEEP ? wave >> 2 : (wave >> 1) & 1, kw = wave & (KP - 1);
    for (int m0 = 0; m0 < (FEW ? n : 1); m0 += 4) {
      const uint16_t* const x = source(m0 + (lane >> 4));
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (m0 > 0) __syncthreads();
      moe_mx4<4, !FEW>(acc, hb, kw, kdim >> 7, KP, sh.slot[wave], [&](int u) {
        return MoeHalf{tiles + (size_t)(u >> 1) * kTileBytes, u & 1, x + (size_t)u * 128};
      });
      __syncthreads();
#pragma unroll
      for (int m = 0; m < 4; ++m) sh.red[wave][m][lane] = acc[m];
      __syncthreads();
      if (wave < n - m0 && wave < 4) {         // wave m: the m-th pick, lane = row of the block
        const size_t s = __builtin_amdgcn_readlane(pick, m0 + wave);
        const int l = lane & 31, w = HALF ? 0 : KP * (lane >> 5);
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < (DEEP ? 1 : 2); ++b)
#pragma unroll
          for (int u = 0; u < KP; ++u) v[b] += sh.red[4 * b + w + u][wave][l] + sh.red[4 * b + w + u][wave][l + 32];
        if constexpr (UP) {
          const float f = silu_mul(v[0], v[1]);
          const size_t at = s * a.inter + (HALF ? 32 : 64) * tile + lane;
          if (!HALF || lane < 32) {
            if (HALF && a.t <= kFewTokens) store_hidden2(a, at, f);
            else a.hidden[at] = (uint16_t)f32_to_bf16_rne(f);
          }
        } else {
          float* const o = a.part + s * a.h + (DEEP ? 64 : 128) * tile + lane;
          o[0] = v[0];
          if constexpr (!DEEP) o[64] = v[1];
        }
      }
    }
    return;
  }
  if constexpr (!FEW) {
    const int t = wave & 3, i = lane & 15;
    auto finish = [&](const f32x4_t (&acc)[2], int count, int m0) {
      if constexpr (F != kDownWide) {          // the second four waves hand their sums over: up, or half of K
        __syncthreads();
        if (blk == 1)
          for (int mt = 0; mt < count; ++mt) sh.other[t][mt][lane] = acc[mt];
        __syncthreads();
        if (blk == 1) return;
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        if (mt >= count) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = m0 + 16 * mt + 4 * (lane >> 4) + e;
          const size_t s = __shfl(pick, m < n ? m : n - 1);
          if (m >= n) continue;
          if constexpr (F == kGateUp)
            a.hidden[s * a.inter + 64 * tile + 16 * t + i] =
                (uint16_t)f32_to_bf16_rne(silu_mul(acc[mt][e], sh.other[t][mt][lane][e]));
          else if constexpr (DEEP)
            a.part[s * a.h + 64 * tile + 16 * t + i] = acc[mt][e] + sh.other[t][mt][lane][e];
          else
            a.part[s * a.h + 128 * tile + 64 * blk + 16 * t + i] = acc[mt][e];
        }
      }
    };
    constexpr int TH = DEEP ? 256 : 512;
    const int th = DEEP ? tid & 255 : tid, row = th >> 5;
    const int steps = DEEP ? (kt_count + 1) >> 1 : kt_count;
    const int count = DEEP && blk == 1 ? kt_count - steps : steps;
    const int kt0 = DEEP && blk == 1 ? min(steps, kt_count - 1) : 0;
    uint8_t* const xs = sh.x[DEEP ? blk : 0];    // two buffers of up to 32 rows
    if (n <= 16) {
      f32x4_t acc[1] = {};
      const uint16_t* xr[512 / TH];
#pragma unroll
      for (int j = 0; j < 512 / TH; ++j) xr[j] = source(row + TH / 32 * j);
      moe_mx16<1, TH>(acc, tiles, t, kt0, count, steps, xr, th, xs);
      const f32x4_t both[2] = {acc[0], acc[0]};
      finish(both, 1, 0);
    }
    for (int m0 = n <= 16 ? n : 0; m0 < n; m0 += 32) {
      f32x4_t acc[2] = {};
      const uint16_t* xr[1024 / TH];
#pragma unroll
      for (int j = 0; j < 1024 / TH; ++j) xr[j] = source(m0 + row + TH / 32 * j);
      if (m0 > 0) __syncthreads();               // the LDS of the tokens before is done with
      moe_mx16<2, TH>(acc, tiles, t, kt0, count, steps, xr, th, xs);
      finish(acc, 2, m0);
    }
  }
}

// ---- combine ----------------------------------------------------------------

__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
  const int t = blockIdx.y, c = blockIdx.x * 1024 + threadIdx.x * 4;
  const float* const l = a.picked + (size_t)t * a.k;
  const float* const part = a.part + (size_t)t * a.k * a.h + min(c, a.h - 4);
  f32x4_t first[8];                      // on their way while the weights are formed
#pragma unroll
  for (int j = 0; j < 8; ++j)
    first[j] = j < a.k ? *reinterpret_cast<const f32x4_t*>(part + (size_t)j * a.h) : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const float total = moe_total(a, t, l);
  if (c >= a.h) return;
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= a.k) continue;
    const float p = expf(l[j] - l[0]) / total;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(p, first[j][e], y[e]);
  }
  for (int j = 8; j < a.k; ++j) {
    const float p = expf(l[j] - l[0]) / total;
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(part + (size_t)j * a.h);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(p, v[e], y[e]);
  }
  const size_t at = (size_t)t * a.h + c;
  if (a.y_f32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.y) + at) = y;
  else
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.y) + at) = u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

// Workspace: each part on 256 bytes.
static int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

int64_t moe_ws_bytes(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t k) {
  const bool few = t <= kFewTokens;
  return up256(t * e * 4) + 2 * up256(t * k * 4) + up256(t * k * inter * (few ? 4 : 2)) +
         (few ? 0 : up256(t * k * h * 4)) + up256(e * 4) + up256(e * 256);
}

hipError_t launch_moe_w4a16(const void* x, int t, int h, const void* router, int e, const void* gate_up,
                            int64_t gate_up_bytes, const void* down, int64_t down_bytes, int inter, int k, int renorm,
                            void* y, int y_f32, void* ws, hipStream_t stream) {
  MoeArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.router = static_cast<const uint16_t*>(router);
  a.gate_up = static_cast<const uint8_t*>(gate_up);
  a.down = static_cast<const uint8_t*>(down);
  a.gate_up_bytes = gate_up_bytes, a.down_bytes = down_bytes;
  a.t = t, a.h = h, a.e = e, a.inter = inter, a.k = k, a.renorm = renorm;
  char* w = static_cast<char*>(ws);
  auto take = [&](int64_t bytes) {
    char* const p = w;
    w += up256(bytes);
    return p;
  };
  a.logits = reinterpret_cast<float*>(take((int64_t)t * e * 4));
  a.picked = reinterpret_cast<float*>(take((int64_t)t * k * 4));
  a.expert_of = reinterpret_cast<int32_t*>(take((int64_t)t * k * 4));
  const bool few = t <= kFewTokens;
  a.hidden = reinterpret_cast<uint16_t*>(take((int64_t)t * k * inter * (few ? 4 : 2)));
  if (!few) a.part = reinterpret_cast<float*>(take((int64_t)t * k * h * 4));
  a.count = reinterpret_cast<int32_t*>(take((int64_t)e * 4));
  a.list = reinterpret_cast<int32_t*>(take((int64_t)e * 256));
  a.y = y, a.y_f32 = y_f32;

  hipError_t st = hipSuccess;
  auto ok = [&] { return (st = hipGetLastError()) == hipSuccess; };
  // Four tokens and an expert a workgroup while they are at most the 8 of 256 threads
  // that a CU holds (64 tokens on 8 experts, h 4096: 48.2 us in all against 51.7; 17 on
  // 64, 2048: 50.6 against 52.8; 64 on 128, 2048 workgroups: 95 both; 64 on 160, 2560: 65
  // against 63.5).
  if (e * ((t + 3) / 4) <= 8 * kCUs)
    hipLaunchKernelGGL(moe_router_gemv_kernel, dim3(e, (t + 3) / 4), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(moe_router_mfma_kernel, dim3((e + 15) / 16, (t + 15) / 16), dim3(1024), 0, stream, a);
  if (!ok()) return st;
  if (t == 1) {
    hipLaunchKernelGGL(moe_gate_up_one_kernel, dim3(inter / 32, k), dim3(1024), 0, stream, a);
    if (!ok()) return st;
    hipLaunchKernelGGL(moe_down_few_kernel, dim3(h / 16), dim3(1024), 0, stream, a);
    return hipGetLastError();
  }
  // Units by experts once few of these are left without tokens: a workgroup then
  // knows its expert without looking for it (17 tokens, 6 of 64 experts of 1024 x
  // 2048: 56 us against 58.7; 16 tokens, 8 of 128: 66 against 63).
  a.direct = 2 * t * k >= 3 * e;
  // Four tokens at a time where few experts have more: up to 2.5 picks per expert on
  // average (17 tokens, 6 of 64 experts of 1024 x 2048: 50.5 us against 55; 7 tokens, 8
  // of 128 of 768 x 4096: 68 against 78; at 2.1 and 2.5 per expert 67 and 71 against 70
  // and 73, at 3 of 16 experts of 3840 x 2560 75.6 against 70.7).
  const bool thin = few || 2 * t * k <= 5 * e;
  // Up to kOwnTokens tokens, ranking takes a workgroup of the gate and up launch about
  // 1 us, which is less than a launch while all of them run at once (thin: 4 tokens, 2 of
  // 8 of 3840 x 1024, 960 workgroups: 18.3 us against 20.3; 6, 4 of 32 of 1280 x 2048, 960:
  // 30.7 against 32.7; 7, 8 of 128 of 768 x 4096, 1344: 64.8 against 63.5; 5, 4 of 16 of
  // 10496 x 2048, 6560: 107 against 89; else: 8, 4 of 8 of 4096 x 2048, 512: 38.1 against
  // 39.3; of 5120, 640: 49.0 against 48.0).
  a.own = t <= kOwnTokens && inter / (thin ? 32 : 64) * (a.direct ? e : t * k) <= (thin ? 4 : 2) * kCUs;
  const int units = a.direct || (!a.own && t * k > e) ? e : t * k;
  if (!a.own) {
    hipLaunchKernelGGL(moe_route_kernel, dim3(e), dim3(512), 0, stream, a);
    if (!ok()) return st;
  }
  if (thin)
    hipLaunchKernelGGL((moe_expert_kernel<kGateUpFew>), dim3(inter / 32, units), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_expert_kernel<kGateUp>), dim3(inter / 64, units), dim3(512), 0, stream, a);
  if (!ok()) return st;
  if (few) {
    hipLaunchKernelGGL(moe_down_few_kernel, dim3(h / 16, t), dim3(1024), 0, stream, a);
    return hipGetLastError();
  }
  // Down in the deep form up to one and a half workgroups per CU, whose second
  // half of the slots the wide form would leave empty (8 of 8 experts of 14336 x 4096
  // hit by 8 tokens, 256 wide workgroups: 150 us against 170 wide; 31 tokens on 8
  // of 6912 x 2048, 128: 64 against 74; 54 on 16 of 6400 x 2560, 320: 134 against 141);
  // above it the wide form copies each activation row for twice the weight rows (60
  // on 16 of 3328 x 4096, 512: 121 us against 129 deep; 16 on 128 of 768 x 2048: 64
  // against 71).
  if (thin)
    hipLaunchKernelGGL((moe_expert_kernel<kDownFew>), dim3(h / 64, units), dim3(512), 0, stream, a);
  else if (2 * (h / 128) * units <= 3 * kCUs)
    hipLaunchKernelGGL((moe_expert_kernel<kDownDeep>), dim3(h / 64, units), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((moe_expert_kernel<kDownWide>), dim3(h / 128, units), dim3(512), 0, stream, a);
  if (!ok()) return st;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((h + 1023) / 1024, t), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
