// kv8_cache.hip -- the paged key/value cache held in 8 bits: appending new
// tokens (kv8_append) and reading sequences back (kv8_read).
//
// A page holds 64 tokens of every key/value head as int8 codes, with one fp32
// scale per 16 tokens, head and keys / values (layout: include/qgemm.h).  For a
// block of 16 tokens that receives new ones, with s_held its scale (0 where
// the block holds no earlier token) and a = max |x| over its new tokens,
//   s = max(s_held, a * (1/127)),
//   held codes  q <- rint(q * (s_held / s))   where s grew,
//   new codes   q  = clamp(rint(x / s), -127, 127)
// in binary32: a block's scale only grows while it holds tokens, so a token is
// requantized at most when a larger one joins its 16.
//
// Mapping of the append: a workgroup owns one page of one head of a sequence
// (nobody else writes it), wave w its block w, so a block's maximum is a
// butterfly within a wave.  Keys: a lane converts 8 channels of one token per
// 16-byte load and stores 8 bytes.  Values are stored channel-major: a lane
// loads the same 8 channels of 4 neighbouring tokens, and has then whole
// dwords (4 tokens of a channel) to store.  A page whose four blocks are all
// written gathers those dwords in LDS and stores 16 bytes per lane (a
// channel's 64 bytes are one run); a page with fewer written blocks (a decode
// step) stores the dwords where they are.
//
// Bound by HBM, 2 bytes read and 1 written per channel: two chunks of 64000 tokens on
// 8 heads of 128 run at 5.05 TB/s, as a large copy does; chunks of 5001 and 16001
// tokens, 129 MB, take 33 us, where a workgroup per page and head is not yet
// several rounds of the card.  One token each for 3 sequences: 5.6 us.
#include <type_traits>

#include "layer_common.h"

namespace qg {

struct AppendArgs {
  Kv8Args c;
  const uint16_t *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
  int64_t max_new;
  uint32_t* status;
};

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// The larger of `m` and the magnitudes in 8 bf16 values, as bf16 patterns in both
// halves: without the sign they order as whole numbers, infinities and NaN last.
__device__ __forceinline__ uint32_t absmax8(const u32x4_t& v, uint32_t m) {
  u16x2_t t = __builtin_bit_cast(u16x2_t, m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i] & 0x7fff7fffu;
    t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2_t, w));
  }
  return __builtin_bit_cast(uint32_t, t);
}

// Codes of four values, packed.  The quotient x / s, correctly rounded, as
// q1 = x y, q = q1 + (x - q1 s) y with y the correctly rounded 1 / s (Markstein's
// step: exact residual by fma); adding 1.5 2^23 rounds it to a whole number, half
// to even, whose low byte is the code.  |x / s| stays below 127.5 since s >= a / 127
// to within 2^-23.  Five instructions a code against about fifteen with the
// divide; scales outside 2^-100 .. 2^100, where a step could leave the normal
// numbers, and NaN (code 0) take that.
template <bool FAST>
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, float s, float y) {
  const float x[4] = {x0, x1, x2, x3};
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FAST) {
      const float q1 = x[i] * y;
      b[i] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q1, s, x[i]), y, q1) + 12582912.0f);
    } else {
      const float q = s > 0.0f ? rintf(x[i] / s) : 0.0f;
      b[i] = (uint32_t)(int)fminf(fmaxf(q, -127.0f), 127.0f);
    }
  }
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                               __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
}

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= ((uint32_t)(int)rintf((float)(int8_t)(w >> (8 * i)) * f) & 0xffu) << (8 * i);
  return o;
}

// The block's new scale from its lanes' maxima (absmax8), the same for the whole
// wave; NaN once anything that is not finite has joined it.  `f` is what the held
// codes are multiplied by.
__device__ __forceinline__ float grow(uint32_t mx, float held, float& f) {
  mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
  for (int o = 1; o < 64; o *= 2) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
  mx = __builtin_amdgcn_readfirstlane(mx);
  f = 1.0f;
  if (mx >= 0x7f80u || held != held) return __uint_as_float(0x7fc00000u);
  const float s = fmaxf(held, bf16_to_f32(mx) * (1.0f / 127.0f));
  if (s > held) f = held / s;
  return s;
}

template <int D>
__global__ __launch_bounds__(256) void kv8_append_kernel(AppendArgs a) {
  constexpr int NK = D / 32;            // 16-byte chunks of keys per lane
  constexpr int CH = D / 8;             // chunks per token
  constexpr int NV = (CH * 4 + 63) / 64;
  // [channel][quad][block], 16 dwords more per 8 channels: the lanes of a store
  // are 8 channels apart, 128 dwords without that
  __shared__ __attribute__((aligned(16))) uint32_t vt[D * 18];
  auto at_vt = [](int d) { return d * 16 + (d >> 3) * 16; };
  const int lane = threadIdx.x & 63;
  const int w = wave_id_uniform();      // block of the page
  const int b = blockIdx.x / a.c.hkv, h = blockIdx.x % a.c.hkv;
  int64_t r0, n;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, n);
  const int64_t total = a.c.lens[b];
  if (n <= 0 || total <= 0) return;
  const int64_t first = total > n ? total - n : 0;   // first token written
  const int64_t shift = r0 - (total - n);            // row of token j: j + shift
  const int64_t len = total - n + min(n, a.max_new); // and the end of those written: rows past max_new are not
  if (len <= first) return;
  const int64_t pi = first / kPage + blockIdx.y;
  if (pi * kPage >= len) return;
  const int page = kv8_page(a.c.table + (size_t)b * a.c.width, a.c.width, a.c.pages, pi);
  if (page < 0) {
    if (a.status && threadIdx.x == 0) atomicOr(a.status, QG_FLAG_PAGE);
    return;
  }
  int8_t* const kc = a.c.codes + kv8_base(page, a.c.hkv, h, D);
  uint32_t* const vc = reinterpret_cast<uint32_t*>(kc + kPage * D);
  float* const sc = a.c.scales + ((size_t)page * a.c.hkv + h) * 8 + w;

  const int64_t t0 = pi * kPage + w * kBlock;    // first token of this wave's block
  const bool touched = t0 < len && t0 + kBlock > first;
  // all four blocks written: the last one is, and the first has no token to leave alone
  const bool whole = pi * kPage >= first / kBlock * kBlock && pi * kPage + 3 * kBlock < len;
  const int lo = first > t0 ? (int)(first - t0) : 0;              // new tokens of the block: [lo, hi)
  const int hi = len - t0 < kBlock ? (int)(len - t0) : kBlock;

  if (touched) {
    const float held_k = lo > 0 ? sc[0] : 0.0f, held_v = lo > 0 ? sc[4] : 0.0f;
    u32x4_t kx[NK], vx[NV][4];
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int c = lane + 64 * i, tok = c / CH;
      kx[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (tok >= lo && tok < hi)
        kx[i] = *reinterpret_cast<const u32x4_t*>(a.k + (t0 + tok + shift) * a.k_ts + h * a.k_hs + c % CH * 8);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + 64 * i, quad = c & 3, ch = c >> 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 4 * quad + e;
        vx[i][e] = u32x4_t{0u, 0u, 0u, 0u};
        if (ch < CH && tok >= lo && tok < hi)
          vx[i][e] = *reinterpret_cast<const u32x4_t*>(a.v + (t0 + tok + shift) * a.v_ts + h * a.v_hs + ch * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < NK; ++i) mk = absmax8(kx[i], mk);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) mv = absmax8(vx[i][e], mv);
    float fk, fv;
    const float sk = grow(mk, held_k, fk), sv = grow(mv, held_v, fv);
    if (a.status && lane == 0 && (sk != sk || sv != sv)) atomicOr(a.status, QG_FLAG_NONFINITE);

    // Keys: held tokens are rewritten only where the scale grew; the rest of
    // a block that held nothing becomes zero.
    auto keys = [&](auto fast) {
      const float y = 1.0f / sk;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int c = lane + 64 * i, tok = c / CH;
        auto four = [&](uint32_t a, uint32_t b) {
          return codes4<decltype(fast)::value>(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u),
                                               __uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u), sk, y);
        };
        u32x2_t* p = reinterpret_cast<u32x2_t*>(kc + (w * kBlock + tok) * D + c % CH * 8);
        if (tok >= lo && (tok < hi || lo == 0)) *p = u32x2_t{four(kx[i].x, kx[i].y), four(kx[i].z, kx[i].w)};
      }
    };
    if (sk >= 0x1p-100f && sk <= 0x1p100f) keys(std::true_type{});
    else keys(std::false_type{});
    if (fk != 1.0f) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int c = lane + 64 * i, tok = c / CH;
        u32x2_t* p = reinterpret_cast<u32x2_t*>(kc + (w * kBlock + tok) * D + c % CH * 8);
        if (tok < lo) {
          const u32x2_t old = *p;
          *p = u32x2_t{rescale4(old.x, fk), rescale4(old.y, fk)};
        }
      }
    }
    // Values: dword (channel, quad) = tokens 4 quad .. + 3 of the block.
    auto values = [&](auto fast) {
      const float y = 1.0f / sv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = lane + 64 * i, quad = c & 3, ch = c >> 2;
        if (ch >= CH) continue;
        // its first `keep` tokens are held, the others new (or zeroed)
        const int q0 = 4 * quad;
        const int keep = lo > q0 ? (lo - q0 < 4 ? lo - q0 : 4) : 0;
        const bool fresh = (lo < q0 + 4 && hi > q0) || lo == 0;
        if (!whole && !fresh && fv == 1.0f) continue;   // nothing of it changes
        const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = 8 * ch + e;
          float x[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t two = vx[i][u][e >> 1];
            x[u] = __uint_as_float((e & 1) ? two & 0xffff0000u : two << 16);
          }
          uint32_t* const p = vc + d * 16 + quad * 4 + w;
          uint32_t o = codes4<decltype(fast)::value>(x[0], x[1], x[2], x[3], sv, y);
          if (lo > 0 && keep) o = (o & ~mask) | (rescale4(*p, fv) & mask);
          if (whole) vt[at_vt(d) + quad * 4 + w] = o;
          else *p = o;
        }
      }
    };
    if (sv >= 0x1p-100f && sv <= 0x1p100f) values(std::true_type{});
    else values(std::false_type{});
    if (lane == 0) {
      sc[0] = sk;
      sc[4] = sv;
    }
  }
  if (!whole) return;                    // uniform over the workgroup
  __syncthreads();
  for (int p = threadIdx.x; p < D * 4; p += 256)
    reinterpret_cast<u32x4_t*>(vc)[p] = *reinterpret_cast<const u32x4_t*>(&vt[at_vt(p >> 2) + (p & 3) * 4]);
}

struct ReadArgs {
  Kv8Args c;
  int64_t max_len;
  void *k, *v;
};

template <bool F32>
__device__ __forceinline__ void store4(void* out, size_t at, uint32_t w, float s) {
  const float x0 = (float)(int8_t)w * s, x1 = (float)(int8_t)(w >> 8) * s, x2 = (float)(int8_t)(w >> 16) * s,
              x3 = (float)(int8_t)(w >> 24) * s;
  if constexpr (F32) {
    const f32x4_t v = {x0, x1, x2, x3};
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at));
  } else {
    const u32x2_t v = {pack_bf16(x0, x1), pack_bf16(x2, x3)};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(out) + at));
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* out, size_t at, u32x2_t w, float s) {
  if constexpr (F32) {
    store4<true>(out, at, w.x, s);
    store4<true>(out, at + 4, w.y, s);
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = (float)(int8_t)(w.x >> (8 * i)) * s;
      x[4 + i] = (float)(int8_t)(w.y >> (8 * i)) * s;
    }
    const u32x4_t v = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + at));
  }
}

// A workgroup reads one page of one head.  Keys: 8 codes per lane.  Values:
// a lane loads 16 bytes (its quad's tokens of all four blocks) of 4
// neighbouring channels, and byte permutes turn each 4 x 4 square round, so
// that 16 lanes store whole 128-byte lines of a token's row.  Stores are
// non-temporal: two bytes written per byte read, 4.9 TB/s against 4.4 (64000
// tokens of two sequences, 8 heads of 128; a large copy moves 5.1).
template <int D, bool F32>
__global__ __launch_bounds__(256) void kv8_read_kernel(ReadArgs a) {
  const int b = blockIdx.x / a.c.hkv, h = blockIdx.x % a.c.hkv;
  const int64_t t0 = (int64_t)blockIdx.y * kPage;
  const int64_t len = a.c.lens[b];
  const int left = (int)(a.max_len - t0 < kPage ? a.max_len - t0 : kPage);              // rows to write
  const int have = len - t0 >= left ? left : len > t0 ? (int)(len - t0) : 0;            // of them with a token
  const int page = have > 0 ? kv8_page(a.c.table + (size_t)b * a.c.width, a.c.width, a.c.pages, blockIdx.y) : 0;
  const size_t row0 = ((size_t)b * a.max_len + t0) * a.c.hkv + h;   // output row of token t: row0 + t hkv
  const float nan = __uint_as_float(0x7fc00000u);
  const int8_t* const kc = a.c.codes + kv8_base(page < 0 ? 0 : page, a.c.hkv, h, D);
  const float* const sc = a.c.scales + ((size_t)(page < 0 ? 0 : page) * a.c.hkv + h) * 8;

  for (int c = threadIdx.x; c < kPage * D / 8; c += 256) {
    const int tok = c / (D / 8), ch = c % (D / 8) * 8;
    if (tok >= left) continue;
    u32x2_t q{0u, 0u};
    float s = 0.0f;
    if (tok < have) {
      q = *reinterpret_cast<const u32x2_t*>(kc + tok * D + ch);
      s = page < 0 ? nan : sc[tok / kBlock];
    }
    store8<F32>(a.k, (row0 + (size_t)tok * a.c.hkv) * D + ch, q, s);
  }
  for (int c = threadIdx.x; c < D; c += 256) {   // (channel quad, token quad)
    const int quad = c & 3, d = c >> 2 << 2;
    u32x4_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = u32x4_t{0u, 0u, 0u, 0u};
      if (have > 0) v[e] = *reinterpret_cast<const u32x4_t*>(kc + kPage * D + (d + e) * 64 + quad * 16);
    }
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
      const float s = page < 0 ? nan : kBlock * blk < have ? sc[4 + blk] : 0.0f;
      // a, b: tokens 0, 1 / 2, 3 of channels 0, 1 and 2, 3
      const uint32_t a01 = __builtin_amdgcn_perm(v[1][blk], v[0][blk], 0x05010400u);   // t0c0 t0c1 t1c0 t1c1
      const uint32_t a23 = __builtin_amdgcn_perm(v[1][blk], v[0][blk], 0x07030602u);
      const uint32_t b01 = __builtin_amdgcn_perm(v[3][blk], v[2][blk], 0x05010400u);
      const uint32_t b23 = __builtin_amdgcn_perm(v[3][blk], v[2][blk], 0x07030602u);
      const uint32_t o[4] = {__builtin_amdgcn_perm(b01, a01, 0x05040100u), __builtin_amdgcn_perm(b01, a01, 0x07060302u),
                             __builtin_amdgcn_perm(b23, a23, 0x05040100u), __builtin_amdgcn_perm(b23, a23, 0x07060302u)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = kBlock * blk + 4 * quad + e;
        if (tok < left)
          store4<F32>(a.v, (row0 + (size_t)tok * a.c.hkv) * D + d, tok < have ? o[e] : 0u, tok < have ? s : 0.0f);
      }
    }
  }
}

hipError_t launch_kv8_append(const Kv8Args& c, const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                             int64_t v_hs, int64_t max_new, uint32_t* status, hipStream_t stream) {
  const AppendArgs a{c, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_ts, k_hs, v_ts, v_hs, max_new,
                     status};
  // max_new tokens that start anywhere in a page reach at most this many pages
  const dim3 grid((uint32_t)(c.b * c.hkv), (uint32_t)((max_new + kPage - 2) / kPage + 1));
  switch (c.d) {
#define QG_APP(D) \
  case D: hipLaunchKernelGGL((kv8_append_kernel<D>), grid, dim3(256), 0, stream, a); break;
    QG_APP(64) QG_APP(128) QG_APP(192) QG_APP(256)
#undef QG_APP
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_kv8_read(const Kv8Args& c, int64_t max_len, void* k, void* v, int f32, hipStream_t stream) {
  const ReadArgs a{c, max_len, k, v};
  const dim3 grid((uint32_t)(c.b * c.hkv), (uint32_t)((max_len + kPage - 1) / kPage));
  switch (c.d) {
#define QG_READ(D)                                                                                      \
  case D:                                                                                               \
    if (f32) hipLaunchKernelGGL((kv8_read_kernel<D, true>), grid, dim3(256), 0, stream, a);             \
    else hipLaunchKernelGGL((kv8_read_kernel<D, false>), grid, dim3(256), 0, stream, a);                \
    break;
    QG_READ(64) QG_READ(128) QG_READ(192) QG_READ(256)
#undef QG_READ
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace qg
