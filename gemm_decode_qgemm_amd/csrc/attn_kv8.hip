// attn_kv8.hip -- attention of a few query rows per sequence over the paged
// 8-bit cache (qg_attn_kv8).
//
//   s_j = scale * q . (kq_j * ks),  o = sum_j softmax(s)_j (vq_j * vs)
// over the tokens j <= position of the row (and > position - window), with ks
// and vs the scales of token j's block; a row with no such token is zero.
//
// One pass with the running maximum m and sum l: for every page of 64 tokens
//   m' = max(m, max s), p = 2^(s - m'), l = l 2^(m - m') + sum p,
//   O  = O 2^(m - m') + sum p v,       o = O / l
// (scores in units of log 2), everything but the products' operands in fp32.
// Operands are bf16: q as given, codes exactly (|q| <= 127), and p * vs
// rounded once, which costs 2^-9 of each term and needs no further pass.
//
// Mapping (gfx950, wave64, v_mfma_f32_16x16x32_bf16):
//  * the rows of one key/value head are its query rows times its query heads;
//    a wave takes 16 NT of them and whole pages, 64 tokens x (K, V), straight
//    from memory to registers, no LDS: S^T = K Q^T, so lane (i, a) =
//    (lane % 16, lane / 16) holds tokens 16 blk + 4a + 0..3 of row i;
//  * exactly those tokens are what the P operand of O^T = V^T P^T wants from
//    that lane, once the order of the contraction over tokens is chosen to
//    match: the cache stores values channel-major with a channel's 64 tokens as
//    [quad a][block][4], so a lane's 16-byte load is its two P operands'
//    partner.  Neither P nor V crosses lanes;
//  * m and l of a row are the same lane column as its O, so rescaling is one
//    factor per lane; it is skipped while no maximum of the wave moved;
//  * a block's scales are wave-uniform (scalar loads);
//  * codes become bf16 by a byte-selecting convert each and one byte permute a
//    pair: 1.5 instructions per code, about a third of the time HBM takes to
//    deliver them at 16 rows.
// A workgroup's waves take pages in turn and join (m, l, O) through LDS; the
// pages of a sequence are further split over workgroups when there are few,
// the partial (m, l, O) joined by a second kernel in a fixed order.
#include "layer_common.h"

namespace qg {

struct AttnArgs {
  Kv8Args c;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  int hq, group, max_q, window, splits, row_tiles;
  float scale_log2;                 // scale * log2(e)
  void* out;
  int out_f32;
  float *part_o, *part_ml;          // [splits][rows * hq][d], [splits][rows * hq][2]
  uint32_t* status;
};

// Value of lane ^ 32, then of lane ^ 16, folded with f.
template <class F>
__device__ __forceinline__ float fold_quads(float v, F f) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

// 8 int8 codes as 8 bf16 (exact: the low half of the fp32 value is zero).
__device__ __forceinline__ bf16x8_t codes8(uint32_t lo, uint32_t hi) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? lo : hi;
    const float x = (float)(int8_t)(w >> (16 * (i & 1))), y = (float)(int8_t)(w >> (16 * (i & 1) + 8));
    o[i] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

constexpr float kNegInf = -__builtin_inff();

template <int D, int NT, int W>
__global__ __launch_bounds__(64 * W) void attn_kv8_kernel(AttnArgs a) {
  constexpr int KC = D / 64;        // 64-channel chunks of a key
  constexpr int DT = D / 16;        // 16-channel tiles of a value
  __shared__ float sm_m[W][16 * NT], sm_l[W][16 * NT];
  __shared__ f32x4_t sm_o[W][DT][64];
  const int lane = threadIdx.x & 63, i = lane & 15, qd = lane >> 4;
  const int wave = wave_id_uniform();
  const int split = blockIdx.x;
  const int h = blockIdx.y / a.row_tiles, rt = blockIdx.y % a.row_tiles, b = blockIdx.z;
  int64_t r0, n64;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, n64);
  const int nq = (int)(n64 < a.max_q ? n64 : a.max_q);
  const int nrows = nq * a.group;
  const int row0 = rt * 16 * NT;
  if (row0 >= nrows) return;
  const int len = max(a.c.lens[b], 0);
  // The last query row is the sequence's last token.
  const int shift = len - (int)n64;                  // position of query row t: shift + t
  const int t_lo = row0 / a.group, t_hi = min(row0 + 16 * NT - 1, nrows - 1) / a.group;
  const int pos_hi = shift + t_hi, pos_lo = shift + t_lo;
  const int tok_end = pos_hi + 1;                    // tokens [tok_beg, tok_end) are seen by some row
  const int tok_beg = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
  int p_beg = 0, p_end = 0;
  if (tok_end > tok_beg) {
    const int first = tok_beg / kPage;
    // a length beyond the table costs one page that is not there
    const int last = (int)min((int64_t)((tok_end - 1) / kPage), a.c.width);
    const int count = last >= first ? last - first + 1 : 0;
    p_beg = first + (int)((int64_t)count * split / a.splits);
    p_end = first + (int)((int64_t)count * (split + 1) / a.splits);
  }

  // Rows of this lane: t = query row, g = head of the group.
  int pos[NT];
  bf16x8_t qf[NT][2 * KC];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 16 * n + i;
    const bool on = r < nrows;
    const int t = r / a.group, g = r - t * a.group;
    pos[n] = on ? shift + t : -1;
    const uint16_t* src = a.q + (r0 + t) * a.q_ts + (int64_t)(h * a.group + g) * a.q_hs + 16 * qd;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        u32x4_t v{0u, 0u, 0u, 0u};
        if (on) v = *reinterpret_cast<const u32x4_t*>(src + 64 * c + 8 * e);
        qf[n][2 * c + e] = __builtin_bit_cast(bf16x8_t, v);
      }
  }

  float m[NT], l[NT];
  f32x4_t o[NT][DT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t* const trow = a.c.table + (size_t)b * a.c.width;
  int next = p_beg + wave < p_end ? kv8_page(trow, a.c.width, a.c.pages, p_beg + wave) : 0;
  for (int p = p_beg + wave; p < p_end; p += W) {
    const int page = __builtin_amdgcn_readfirstlane(next);
    if (p + W < p_end) next = kv8_page(trow, a.c.width, a.c.pages, p + W);
    const int held = page < 0 ? 0 : page;            // reads stay inside; its scales become NaN below
    const int8_t* const kc = a.c.codes + kv8_base(held, a.c.hkv, h, D);
    const float* const sc = a.c.scales + ((size_t)held * a.c.hkv + h) * 8;
    u32x4_t kr[4][KC], vr[DT];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk)
#pragma unroll
      for (int c = 0; c < KC; ++c)
        kr[blk][c] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(kc + (16 * blk + i) * D + 64 * c + 16 * qd));
#pragma unroll
    for (int t = 0; t < DT; ++t)
      vr[t] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(kc + kPage * D + 1024 * t + 64 * i + 16 * qd));
    float ks[4], vs[4];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
      ks[blk] = page < 0 ? __uint_as_float(0x7fc00000u) : sc[blk] * a.scale_log2;
      vs[blk] = sc[4 + blk];
    }
    if (page < 0 && a.status && lane == 0) atomicOr(a.status, QG_FLAG_PAGE);
    const int j0 = p * kPage;
    const bool edge = j0 + kPage - 1 > pos_lo || (a.window > 0 && j0 <= pos_hi - a.window);   // uniform

    f32x4_t s[NT][4];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][blk] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const bf16x8_t k0 = codes8(kr[blk][c][0], kr[blk][c][1]), k1 = codes8(kr[blk][c][2], kr[blk][c][3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[n][2 * c], s[n][blk], 0, 0, 0);
          s[n][blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[n][2 * c + 1], s[n][blk], 0, 0, 0);
        }
      }
    }
    bf16x8_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = kNegInf;
#pragma unroll
      for (int blk = 0; blk < 4; ++blk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[n][blk][e] * ks[blk];
          if (edge) {
            const int j = j0 + 16 * blk + 4 * qd + e;
            v = j <= pos[n] && (a.window <= 0 || j > pos[n] - a.window) ? v : kNegInf;
          }
          s[n][blk][e] = v;
          mx = fmaxf(mx, v);
        }
      mx = fold_quads(mx, [](float x, float y) { return fmaxf(x, y); });
      const float m_new = fmaxf(m[n], mx);
      const float base = m_new == kNegInf ? 0.0f : m_new;   // nothing seen yet: every p is 0
      if (__ballot(m_new > m[n]) != 0) {
        const float f = __builtin_amdgcn_exp2f(m[n] - base);
        l[n] *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][t][e] *= f;
        m[n] = m_new;
      }
      u32x4_t w[2];
      float sum = 0.0f;
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) {
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[n][blk][e] - base);
          sum += x;
          pv[e] = x * vs[blk];
          // a scale that holds a NaN, or was never written, stays out of rows that do not see its block
          if (edge) pv[e] = s[n][blk][e] == kNegInf ? 0.0f : pv[e];
        }
        w[blk >> 1][2 * (blk & 1)] = pack_bf16(pv[0], pv[1]);
        w[blk >> 1][2 * (blk & 1) + 1] = pack_bf16(pv[2], pv[3]);
      }
      l[n] += sum;
      pf[n][0] = __builtin_bit_cast(bf16x8_t, w[0]);
      pf[n][1] = __builtin_bit_cast(bf16x8_t, w[1]);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const bf16x8_t v0 = codes8(vr[t][0], vr[t][1]), v1 = codes8(vr[t][2], vr[t][3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pf[n][0], o[n][t], 0, 0, 0);
        o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pf[n][1], o[n][t], 0, 0, 0);
      }
    }
  }

  // Join the waves: M = max m, each wave's O and l times 2^(m - M), added in wave order.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] = fold_quads(l[n], [](float x, float y) { return x + y; });
    if (qd == 0) {
      sm_m[wave][16 * n + i] = m[n];
      sm_l[wave][16 * n + i] = l[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float mm = kNegInf, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) mm = fmaxf(mm, sm_m[w][16 * n + i]);
    const float base = mm == kNegInf ? 0.0f : mm;
#pragma unroll
    for (int w = 0; w < W; ++w) ll += sm_l[w][16 * n + i] * __builtin_amdgcn_exp2f(sm_m[w][16 * n + i] - base);
    const float f = __builtin_amdgcn_exp2f(m[n] - base);
    if (n > 0) __syncthreads();
#pragma unroll
    for (int t = 0; t < DT; ++t)
      sm_o[wave][t][lane] = f32x4_t{o[n][t][0] * f, o[n][t][1] * f, o[n][t][2] * f, o[n][t][3] * f};
    __syncthreads();
    const int r = row0 + 16 * n + i;
    const int t = r / a.group, g = r - t * a.group;
    const int64_t row = (r0 + t) * a.hq + h * a.group + g;     // row of the output
    const bool on = r < nrows;
    for (int dt = wave; dt < DT; dt += W) {
      f32x4_t v = sm_o[0][dt][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        const f32x4_t u = sm_o[w][dt][lane];
        v = f32x4_t{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
      }
      if (!on) continue;
      const int d = 16 * dt + 4 * qd;
      if (a.splits > 1) {
        if (mm != kNegInf || ll != 0.0f)
          *reinterpret_cast<f32x4_t*>(a.part_o + ((size_t)split * a.c.rows * a.hq + row) * D + d) = v;
      } else {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        const f32x4_t y{v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
        if (a.out_f32)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (size_t)row * D + d) = y;
        else
          *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + (size_t)row * D + d) =
              u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      }
    }
    if (a.splits > 1 && on && wave == 0 && qd == 0) {
      float* const ml = a.part_ml + ((size_t)split * a.c.rows * a.hq + row) * 2;
      ml[0] = mm;
      ml[1] = ll;
    }
  }
}

// The splits of one row and head: a workgroup of 4 waves, each a quarter of
// the splits, joined in order.  Rows that belong to no sequence are left as
// they are.
template <int D>
__global__ __launch_bounds__(256) void attn_kv8_join_kernel(AttnArgs a) {
  constexpr int E = D / 64;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
  const int lane = threadIdx.x & 63, wave = wave_id_uniform();
  // (sequence, query row, head)
  const int b = blockIdx.z, t = blockIdx.y, hd = blockIdx.x;
  int64_t r0, n;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, n);
  if (t >= n) return;
  const size_t total = (size_t)a.c.rows * a.hq, row = (size_t)(r0 + t) * a.hq + hd;
  float m = kNegInf, l = 0.0f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  const int s0 = a.splits * wave / 4, s1 = a.splits * (wave + 1) / 4;
  for (int s = s0; s < s1; ++s) {
    const float* ml = a.part_ml + ((size_t)s * total + row) * 2;
    const float ms = ml[0], ls = ml[1];
    if (ms == kNegInf && ls == 0.0f) continue;           // the split saw nothing and wrote no O
    const float* po = a.part_o + ((size_t)s * total + row) * D + lane * E;
    const float m_new = fmaxf(m, ms), base = m_new == kNegInf ? 0.0f : m_new;
    const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(ms - base);
    m = m_new;
    l = l * f + ls * g;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + po[e] * g;
  }
  if (lane == 0) {
    sm_m[wave] = m;
    sm_l[wave] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[wave][lane * E + e] = o[e];
  __syncthreads();
  if ((int)threadIdx.x >= D) return;
  float mm = kNegInf, ll = 0.0f, v = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm_m[w]);
  const float base = mm == kNegInf ? 0.0f : mm;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = __builtin_amdgcn_exp2f(sm_m[w] - base);
    ll += sm_l[w] * f;
    v += sm_o[w][threadIdx.x] * f;
  }
  v = ll == 0.0f ? 0.0f : v / ll;
  if (a.out_f32)
    static_cast<float*>(a.out)[row * D + threadIdx.x] = v;
  else
    static_cast<uint16_t*>(a.out)[row * D + threadIdx.x] = (uint16_t)f32_to_bf16_rne(v);
}

// Row tiles a wave takes at once: two where a head has more than 16 rows, so
// that a page's codes are converted once for both.
int attn_kv8_nt(int64_t rows_per_head) { return rows_per_head > 16 ? 2 : 1; }

// Splits of a sequence's pages over workgroups.
int attn_kv8_splits(int64_t b, int hkv, int64_t rows_per_head, int64_t max_len, int window, int64_t max_q) {
  const int nt = attn_kv8_nt(rows_per_head);
  const int64_t units = b * hkv * ((rows_per_head + 16 * nt - 1) / (16 * nt));
  int64_t seen = max_len;
  if (window > 0 && window + max_q < seen) seen = window + max_q;
  const int64_t pages = (seen + kPage - 1) / kPage;
  int64_t s = (2 * kCUs + units - 1) / units;
  const int64_t most = (pages + 3) / 4;                 // a page for every wave
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s > 256 ? 256 : s);
}

template <int D, int NT>
static hipError_t launch_attn_t(const AttnArgs& a, hipStream_t stream) {
  constexpr int W = 4;
  hipLaunchKernelGGL((attn_kv8_kernel<D, NT, W>), dim3(a.splits, a.row_tiles * a.c.hkv, a.c.b), dim3(64 * W), 0,
                     stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_kv8_join_kernel<D>), dim3(a.hq, a.max_q, a.c.b), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_attn_kv8(const Kv8Args& c, const void* q, int64_t q_ts, int64_t q_hs, int hq, int max_q, int window,
                           float scale, void* out, int out_f32, int splits, float* part, uint32_t* status,
                           hipStream_t stream) {
  const int group = hq / c.hkv;
  const int64_t rows_per_head = (int64_t)max_q * group;
  const int nt = attn_kv8_nt(rows_per_head);
  AttnArgs a{c, static_cast<const uint16_t*>(q), q_ts, q_hs, hq, group, max_q, window, splits,
             (int)((rows_per_head + 16 * nt - 1) / (16 * nt)), scale * 1.44269504088896340736f, out, out_f32,
             part, part ? part + (size_t)splits * c.rows * hq * c.d : nullptr, status};
  switch (c.d * 4 + nt) {
#define QG_ATTN(D, NT) \
  case D * 4 + NT: return launch_attn_t<D, NT>(a, stream);
    QG_ATTN(64, 1) QG_ATTN(64, 2) QG_ATTN(128, 1) QG_ATTN(128, 2) QG_ATTN(192, 1) QG_ATTN(192, 2)
    QG_ATTN(256, 1) QG_ATTN(256, 2)
#undef QG_ATTN
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
