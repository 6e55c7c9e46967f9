// moe_w4a16.hip -- a whole mixture-of-experts layer for up to 64 tokens on
// packed INT4 group-32 experts (qg_moe_w4a16).
//
//   l = x Wr^T;  the top k experts of a token (ties: the lowest index);
//   p = softmax over the picked logits, or over all of them;
//   y = sum over the picked e of p_e W2_e (silu(Wg_e x) * (Wu_e x))
// with the products of qgemm_w4a16: exact bf16 (128 + q) times bf16
// activations, fp32 sums, the group scale and -(128 + zp) times the group sum
// of x applied per group in fp32.  The hidden activation is rounded to bf16
// once, as the second product's operand; all else is fp32.
//
// Four launches, no atomics (bit-identical repeats):
//  1. router: logits in fp32.
//  2. gate and up: a workgroup owns 32 hidden columns of one expert: four
//     waves the 32 gate rows, four the 32 up rows, each a quarter of K; the
//     two sums meet in LDS and leave as silu(g) u per (token, pick).
//  3. down: the same kernel on two neighbouring 32-row blocks, fp32 results
//     per (token, pick).
//  4. combine: the weighted sum over a token's picks, in order of rank.
// No launch plans the routing: each workgroup of 2 and 3 ranks the logits it
// needs (a few KB from L2).  The rank of expert e for a token is the number of
// experts before it, so "which tokens picked e" takes one ballot per 64
// experts and token, and a token's pick number is that rank.  The grid has
// min(t k, e) units: one per pick, where a pick that shares its expert with
// an earlier token leaves at once, or one per expert.
//
// Two forms of the product, chosen by the tokens the workgroup finds:
//  * up to 4: the 4x4x4 sixteen-block matrix instruction with lane = weight row
//    (the mapping of gemv_w4a16_mx4.hip);
//  * more: 16x16x32 with 16 MT tokens at a time (the mapping of the register
//    form of gemm_w4a16_mfma.hip), weights read again per 16 MT tokens (L2).
#include "layer_common.h"
#include "w4_common.h"

namespace qg {

struct MoeArgs {
  const uint16_t *x, *router;
  const uint8_t *gate_up, *down;
  size_t gate_up_bytes, down_bytes;   // per expert
  int t, h, e, inter, k, renorm, by_pick;
  float* logits;                      // [t, e]
  float* picked;                      // [t * k] logits in order of rank
  uint16_t* hidden;                   // [t * k, inter]
  float* part;                        // [t * k, h]
  void* y;
  int y_f32;
};

// ---- 1: router ---------------------------------------------------------------

// Up to 4 tokens: a wave per expert.
__global__ __launch_bounds__(256) void moe_router_gemv_kernel(MoeArgs a) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + wave_id_uniform();
  if (e >= a.e) return;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c = lane * 8; c < a.h; c += 512) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(a.router + (size_t)e * a.h + c);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m >= a.t) continue;
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(a.x + (size_t)m * a.h + c);
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
    if (m < a.t && lane == 0) a.logits[(size_t)m * a.e + e] = acc[m];
  }
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
#pragma unroll 4
  for (int c = wave * 32; c < a.h; c += 512)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(x + c)),
                                                  __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(w + c)),
                                                  acc, 0, 0, 0);
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

// A logit as an unsigned number of the same order; NaN is above all, -0 is 0.
__device__ __forceinline__ uint32_t order_key(float l) {
  l += 0.0f;
  const uint32_t u = __float_as_uint(l);
  if (l != l) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct MoePlan {
  uint32_t key[512];
  int count[512];
  int rank[64];
  int tok[64], slot[64];   // tokens of the expert in order, and their picks t k + rank
  int expert;
};

// The expert of this workgroup's unit and its tokens; returns how many (0:
// nothing to do).  Workgroups of 512 threads.
__device__ int moe_plan(const MoeArgs& a, int unit, MoePlan& p) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  int first = -1, expert = unit;
  if (a.by_pick) {
    first = unit / a.k;
    const int want = unit - first * a.k;
    if (tid < a.e) p.key[tid] = order_key(a.logits[(size_t)first * a.e + tid]);
    p.count[tid] = 0;
    __syncthreads();
    int width = 64;
    while (width < a.e) width *= 2;
    const int parts = 512 / width, e = tid & (width - 1), part = tid / width;
    if (e < a.e) {
      const uint32_t mine = p.key[e];
      int c = 0;
      for (int o = a.e * part / parts; o < a.e * (part + 1) / parts; ++o)
        c += p.key[o] > mine || (p.key[o] == mine && o < e);
      atomicAdd(&p.count[e], c);
    }
    __syncthreads();
    if (tid < a.e && p.count[tid] == want) p.expert = tid;
    __syncthreads();
    expert = p.expert;
  }
  for (int t = wave; t < a.t; t += 8) {
    const float* row = a.logits + (size_t)t * a.e;
    const uint32_t mine = order_key(row[expert]);
    int c = 0;
    for (int o = lane; o - lane < a.e; o += 64) {
      const uint32_t u = o < a.e ? order_key(row[o]) : 0u;
      c += __popcll(__ballot(o < a.e && (u > mine || (u == mine && o < expert))));
    }
    if (lane == 0) p.rank[t] = c;
  }
  __syncthreads();
  const bool sel = lane < a.t && p.rank[lane < a.t ? lane : 0] < a.k;
  const uint64_t mask = __ballot(sel);
  const int n = __popcll(mask);
  if (wave == 0 && sel) {
    const int at = __popcll(mask & (((uint64_t)1 << lane) - 1));
    p.tok[at] = lane;
    p.slot[at] = lane * a.k + p.rank[lane];
  }
  if (tid == 0) p.expert = expert;
  __syncthreads();
  return a.by_pick && n > 0 && p.tok[0] != first ? 0 : n;
}

// ---- 2 and 3: the experts' products ------------------------------------------

constexpr int kMoeXRow = 288;     // LDS bytes of a token's 128 k (two runs of 128, 16 apart)
constexpr int kMoeXPair = 144;

union MoeShared {
  struct {
    uint8_t x[8][4 * kMoeXRow];
    float sum[8][4][4];           // group sums of x: [wave][group][token]
  } s;
  f32x4_t red[8][2][64];
  float red4[8][4][64];
};

// acc[m] += dequant(W)[row] . x_m over this wave's half tiles, for up to 4 rows
// of activations; lane l holds row l & 31 and the group pair l >> 5.
__device__ __forceinline__ void moe_mx4(float (&acc)[4], const uint8_t* tiles, int row, int halves, int kw,
                                        const uint16_t* xrow, uint8_t* slot, float (*sums)[4]) {
  using L = W4Layout<false>;
  const int lane = threadIdx.x & 63, lg = lane >> 5, sm = lane >> 4, sc = lane & 15;
  const int swr = sm * kMoeXRow + 16 * sc + (sc >= 8 ? 16 : 0);
  const int srd = (lane & 3) * kMoeXRow + lg * kMoeXPair;
  const uint32_t mask_s = __builtin_amdgcn_readfirstlane(0x000F000Fu);
  uint32_t magic_v = 0x43004300u;
  asm volatile("" : "+v"(magic_v));
  uint32_t ones_v = 0x3f803f80u;
  asm volatile("" : "+v"(ones_v));
  auto load = [&](Half32Regs& r, u32x4_t& xv, int hs) {
    L::load(r, tiles + (size_t)(hs >> 1) * L::kTile, hs & 1, lg, row);
    xv = *reinterpret_cast<const u32x4_t*>(xrow + (size_t)hs * 128 + 8 * sc);
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
    *reinterpret_cast<u32x4_t*>(slot + swr) = xv;
    if ((sc & 3) == 0) sums[sc >> 2][sm] = xp;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      u32x4_t xa[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) xa[q] = *reinterpret_cast<const u32x4_t*>(slot + srd + 64 * jj + 16 * q);
      f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const u32x2_t b = {code_pair(r.c[jj][t >> 1], 2 * (t & 1), mask_s, magic_v),
                           code_pair(r.c[jj][t >> 1], 2 * (t & 1) + 1, mask_s, magic_v)};
        const u32x4_t xq = xa[t >> 1];
        d = mfma_4x4x4((t & 1) ? u32x2_t{xq.z, xq.w} : u32x2_t{xq.x, xq.y}, b, d);
      }
      const float s = L::scale(r.sc, jj, 1.0f);
      const f32x4_t xg = *reinterpret_cast<const f32x4_t*>(&sums[2 * lg + jj][0]);
      const float zb = (float)(L::zero(r, jj) | 0x80u);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = __builtin_fmaf(s, __builtin_fmaf(-zb, xg[m], d[m]), acc[m]);
    }
  };
  // two register sets in turn: the next half tile's loads in flight while
  // this one computes
  int hs = kw;
  if (hs >= halves) return;
  Half32Regs ra, rb;
  u32x4_t xa, xb;
  load(ra, xa, hs);
  __builtin_amdgcn_sched_barrier(0);
  while (true) {
    if (hs + 4 >= halves) { compute(ra, xa); break; }
    load(rb, xb, hs + 4);
    __builtin_amdgcn_sched_barrier(0);
    compute(ra, xa);
    hs += 4;
    if (hs + 4 >= halves) { compute(rb, xb); break; }
    load(ra, xa, hs + 4);
    __builtin_amdgcn_sched_barrier(0);
    compute(rb, xb);
    hs += 4;
  }
}

template <int MT>
struct MoeUnit {
  u32x4_t w[2];           // chunk of group a, row 16t + i
  u32x2_t sc;             // row l & 31: the half tile's 4 scales
  uint32_t zw;            // and zero points
  u32x4_t x[MT][4];       // x[token 16 mt + i][32 g + 8 a ..]
};

// Two copies of a register whose 16-lane rows hold (r0, r1, r0, r1): row 0 and row 1 of it in every lane row.
__device__ __forceinline__ u32x2_t spread2(uint32_t v) {
  const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return u32x2_t{s[0], s[1]};
}

// The same for 16 MT rows of activations: acc[t][mt][e] is weight row 16t + i
// and activation row 16 mt + 4a + e.
template <int MT>
__device__ __forceinline__ void moe_mx16(f32x4_t (&acc)[2][MT], const uint8_t* tiles, int hb, int halves, int kw,
                                         const uint16_t* const (&xrow)[MT]) {
  const int lane = threadIdx.x & 63, i = lane & 15, a = lane >> 4, row = 32 * hb + (lane & 31);
  const uint32_t mask_s = __builtin_amdgcn_readfirstlane(0x000F000Fu);
  uint32_t magic_v = 0x43004300u;
  asm volatile("" : "+v"(magic_v));
  uint32_t one2 = 0x3f803f80u;
  asm volatile("" : "+v"(one2));
  const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{one2, one2, one2, one2});
  const f32x4_t zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
  auto load = [&](MoeUnit<MT>& u, int hs) {
    const BufView v(tiles + (size_t)(hs >> 1) * kTileBytes, kTileBytes);
    const int half = hs & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      u.w[t] = v.b128<true>((uint32_t)((4 * half + a) * kTileRows + 32 * hb + 16 * t + i) * 16u);
    u.sc = v.b64((uint32_t)(kScaleOff + row * 16 + 8 * half));
    u.zw = v.b16((uint32_t)(kZeroOff + row * 4 + 2 * half));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        u.x[mt][g] = *reinterpret_cast<const u32x4_t*>(xrow[mt] + (size_t)hs * 128 + 32 * g + 8 * a);
  };
  auto compute = [&](MoeUnit<MT>& u) {
    transpose_rows4(u.w[0]);
    transpose_rows4(u.w[1]);
    const u32x2_t s0 = spread2(u.sc.x), s1 = spread2(u.sc.y), zz = spread2(u.zw);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4_t xg[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        xg[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, u.x[mt][g]), ones, zero4, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4_t bp;
#pragma unroll
        for (int e = 0; e < 4; ++e) bp[e] = code_pair(u.w[t][g], e, mask_s, magic_v);
        const uint32_t sw = g < 2 ? s0[t] : s1[t];
        const float s = fp16_to_f32((sw >> (16 * (g & 1))) & 0xffffu);
        const float zb = (float)(((zz[t] >> (4 * g)) & 15u) | 0x80u);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const f32x4_t p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, u.x[mt][g]),
                                                                    __builtin_bit_cast(bf16x8_t, bp), zero4, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[t][mt][e] = __builtin_fmaf(s, __builtin_fmaf(-zb, xg[mt][e], p[e]), acc[t][mt][e]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // a group's products are not all live at once
    }
  };
  int hs = kw;
  if (hs >= halves) return;
  MoeUnit<MT> ua, ub;
  load(ua, hs);
  __builtin_amdgcn_sched_barrier(0);
  while (true) {
    if (hs + 4 >= halves) { compute(ua); break; }
    load(ub, hs + 4);
    __builtin_amdgcn_sched_barrier(0);
    compute(ua);
    hs += 4;
    if (hs + 4 >= halves) { compute(ub); break; }
    load(ua, hs + 4);
    __builtin_amdgcn_sched_barrier(0);
    compute(ub);
    hs += 4;
  }
}

// silu(g) u as bf16.
__device__ __forceinline__ uint16_t silu_mul(float g, float u) {
  return (uint16_t)f32_to_bf16_rne(g / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g)) * u);
}

// SMALL: no expert has more than 4 tokens (at most 4 tokens in all).
template <bool DOWN, bool SMALL>
__global__ __launch_bounds__(512) void moe_expert_kernel(MoeArgs a) {
  __shared__ MoePlan plan;
  __shared__ __attribute__((aligned(16))) MoeShared sh;
  const int n = moe_plan(a, blockIdx.y, plan);
  if (n == 0) return;                        // uniform over the workgroup
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int blk = wave >> 2, kw = wave & 3;
  const int tile = blockIdx.x, expert = plan.expert;
  if (!DOWN && tile == 0 && tid < n) {
    const int t = plan.tok[tid];
    a.picked[plan.slot[tid]] = a.logits[(size_t)t * a.e + expert];
  }
  const int kdim = DOWN ? a.inter : a.h, halves = kdim >> 7;
  // gate_up: gate rows 32 tile.. and up rows inter + 32 tile..; down: rows
  // 64 tile.. and 64 tile + 32..
  const int rb = DOWN ? tile : (tile >> 1) + blk * (a.inter >> 6);
  const int hb = DOWN ? blk : tile & 1;
  const uint8_t* const tiles = (DOWN ? a.down + expert * a.down_bytes : a.gate_up + expert * a.gate_up_bytes) +
                               (size_t)rb * (kdim >> 8) * kTileBytes;
  auto source = [&](int m) {                 // activation row of the expert's m-th token
    m = m < n ? m : n - 1;
    return DOWN ? a.hidden + (size_t)plan.slot[m] * a.inter : a.x + (size_t)plan.tok[m] * a.h;
  };
  // Row r (of 32) of block b for the m-th token: v0, v1 the sums of both blocks.
  auto store = [&](int m, int r, float v0, float v1) {
    const size_t slot = plan.slot[m];
    if constexpr (DOWN) {
      float* const o = a.part + slot * a.h + 64 * tile + r;
      o[0] = v0;
      o[32] = v1;
    } else {
      a.hidden[slot * a.inter + 32 * tile + r] = silu_mul(v0, v1);
    }
  };

  if (SMALL || n <= 4) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    moe_mx4(acc, tiles, 32 * hb + (lane & 31), halves, kw, source(lane >> 4), sh.s.x[wave], sh.s.sum[wave]);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 4; ++m) sh.red4[wave][m][lane] = acc[m];
    __syncthreads();
    if (tid < 32 * n) {
      const int m = tid >> 5, r = tid & 31;
      float v[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        v[b] = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) v[b] += sh.red4[4 * b + w][m][r] + sh.red4[4 * b + w][m][r + 32];
      }
      store(m, r, v[0], v[1]);
    }
    return;
  }
  if constexpr (!SMALL) {
    const int i = lane & 15;
    auto finish = [&](const f32x4_t (&acc0)[2], int m0) {   // tokens m0 .. m0 + 15
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 2; ++t) sh.red[wave][t][lane] = acc0[t];
      __syncthreads();
      if (tid < 128) {
        const int t = tid >> 6, l = tid & 63;
        f32x4_t v[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          v[b] = sh.red[4 * b][t][l];
#pragma unroll
          for (int w = 1; w < 4; ++w) {
            const f32x4_t u = sh.red[4 * b + w][t][l];
            v[b] = f32x4_t{v[b][0] + u[0], v[b][1] + u[1], v[b][2] + u[2], v[b][3] + u[3]};
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = m0 + 4 * (l >> 4) + e;
          if (m < n) store(m, 16 * t + (l & 15), v[0][e], v[1][e]);
        }
      }
    };
    if (n <= 16) {
      f32x4_t acc[2][1] = {};
      const uint16_t* const rows[1] = {source(i)};
      moe_mx16<1>(acc, tiles, hb, halves, kw, rows);
      const f32x4_t one[2] = {acc[0][0], acc[1][0]};
      finish(one, 0);
    } else {
      for (int m0 = 0; m0 < n; m0 += 32) {
        f32x4_t acc[2][2] = {};
        const uint16_t* const rows[2] = {source(m0 + i), source(m0 + 16 + i)};
        moe_mx16<2>(acc, tiles, hb, halves, kw, rows);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const f32x4_t one[2] = {acc[0][mt], acc[1][mt]};
          finish(one, m0 + 16 * mt);
        }
      }
    }
  }
}

// ---- 4: combine ----------------------------------------------------------------

__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
  const int t = blockIdx.y, c = blockIdx.x * 1024 + threadIdx.x * 4;
  const int lane = threadIdx.x & 63;
  const float* const l = a.picked + (size_t)t * a.k;
  const float top = l[0];                      // rank 0: the largest
  float total = 0.0f;
  if (a.renorm) {
    for (int j = 0; j < a.k; ++j) total += expf(l[j] - top);
  } else {
    for (int e = lane; e < a.e; e += 64) total += expf(a.logits[(size_t)t * a.e + e] - top);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
  }
  if (c >= a.h) return;
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < a.k; ++j) {
    const float p = expf(l[j] - top) / total;
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.part + ((size_t)t * a.k + j) * a.h + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(p, v[e], y[e]);
  }
  const size_t at = (size_t)t * a.h + c;
  if (a.y_f32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.y) + at) = y;
  else
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.y) + at) = u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

// Workspace: logits, picked logits, hidden, partial results, each on 256 bytes.
static int64_t up256(int64_t n) { return (n + 255) & ~(int64_t)255; }

int64_t moe_ws_bytes(int64_t t, int64_t h, int64_t e, int64_t inter, int64_t k) {
  return up256(t * e * 4) + up256(t * k * 4) + up256(t * k * inter * 2) + up256(t * k * h * 4);
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
  a.by_pick = t * k < e;
  char* w = static_cast<char*>(ws);
  a.logits = reinterpret_cast<float*>(w);
  w += up256((int64_t)t * e * 4);
  a.picked = reinterpret_cast<float*>(w);
  w += up256((int64_t)t * k * 4);
  a.hidden = reinterpret_cast<uint16_t*>(w);
  w += up256((int64_t)t * k * inter * 2);
  a.part = reinterpret_cast<float*>(w);
  a.y = y, a.y_f32 = y_f32;

  if (t <= 4)
    hipLaunchKernelGGL(moe_router_gemv_kernel, dim3((e + 3) / 4), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(moe_router_mfma_kernel, dim3((e + 15) / 16, (t + 15) / 16), dim3(1024), 0, stream, a);
  hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  const int units = a.by_pick ? t * k : e;
  const dim3 g1(inter / 32, units), g2(h / 64, units);
  if (t <= 4) {
    hipLaunchKernelGGL((moe_expert_kernel<false, true>), g1, dim3(512), 0, stream, a);
    if ((st = hipGetLastError()) != hipSuccess) return st;
    hipLaunchKernelGGL((moe_expert_kernel<true, true>), g2, dim3(512), 0, stream, a);
  } else {
    hipLaunchKernelGGL((moe_expert_kernel<false, false>), g1, dim3(512), 0, stream, a);
    if ((st = hipGetLastError()) != hipSuccess) return st;
    hipLaunchKernelGGL((moe_expert_kernel<true, false>), g2, dim3(512), 0, stream, a);
  }
  if ((st = hipGetLastError()) != hipSuccess) return st;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((h + 1023) / 1024, t), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
