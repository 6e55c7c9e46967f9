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
// (scores in units of log 2, m rounded up to a whole number so that every rescaling is
// by a power of two), everything but the products' operands in fp32.
// Operands are fp16, which costs fewer instructions than bf16 and rounds less:
//  * a code q becomes 1024 + (q + 128) by one byte permute a pair (0x6400 |
//    byte), exactly.  Keys stay so: the accumulator starts at -1152 sum(q) of the
//    row, and the rounding this costs (2^-24 of 1152 |sum q| against a score of
//    some 40 sqrt(d) |q|) is below 2^-15 of the score.  Values, which are summed
//    over a whole cache, have the 1152 taken off again, exactly (packed add);
//  * a query row is scaled by a power of two to a largest channel in [2^7,
//    2^8), where its 8 significant bits fit exactly;
//  * p * vs is taken relative to the largest one that the row itself has seen so far,
//    put at 2^13 .. 2^15, so it keeps 11 bits down to 2^-27 of that, and 2^-38 of that
//    below.  The power of two is a state of the row like m (one for all rows of a
//    tile, from the scales alone, let a block that a row does not see, or hardly
//    weighs, round the row's own products away).
// As bf16 the same products took 1.5 instructions per code and p * vs had to be
// two operands for this accuracy: 32 sequences of 4096 tokens on 32 / 8 heads of
// 128 in two splits ran 60 us, and 46 once in fp16.  Today they take 48 us (5.6 TB/s),
// 46 (5.85) in one split, which a caller who knows that they are equal can ask for.
//
// Mapping (gfx950, wave64, v_mfma_f32_16x16x32_f16):
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
//  * a block's scales are wave-uniform and read by scalar loads.
// A workgroup's waves take pages in turn and join (m, l, O) through LDS (or, with
// many rows, each a row tile through all pages and join nothing); the
// pages of a sequence are further split over workgroups when there are few,
// the partial (m, l, O) joined by a second kernel in a fixed order.
#include <algorithm>

#include "layer_common.h"

namespace qg {

struct AttnArgs {
  Kv8Args c;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  int hq, group, max_q, window, splits, chunk, row_tiles;
  uint32_t magic;                   // floor(2^32 / group)
  float scale_log2;                 // scale * log2(e)
  void* out;
  int out_f32;
  float *part_o, *part_ml;          // [splits][rows * hq][d], [splits][rows * hq][2]; balanced: see slots
  int slots;                        // > 0: splits are shared out by length, [slots][max_q * hq] partial results
  int even;                         // then: the splits of each sequence where all are about as long,
  int32_t* plan;                    // and [b][2]: a sequence's first slot and their number
  uint32_t* status;
};

// r / group for 0 <= r < 2^31: the product with floor(2^32 / group) is at most
// one short.
__device__ __forceinline__ int group_of(const AttnArgs& a, int r) {
  if (a.group == 1) return r;       // (2^32 does not fit the word)
  const int q = (int)__umulhi((uint32_t)r, a.magic);
  return q + (r - q * a.group >= a.group ? 1 : 0);
}

constexpr int kMinExp = -107;       // products p * vs below 2^-107 are taken relative to that
constexpr int kTopExp = 14;         // the largest is put below 2^(kTopExp + 1)

// Value of lane ^ 32, then of lane ^ 16, folded with f.
template <class F>
__device__ __forceinline__ float fold_quads(float v, F f) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(x[0]), __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(y[0]), __uint_as_float(y[1]));
}

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// 8 int8 codes as fp16, plus 1152 where BIAS: with the sign bit flipped a code
// q is the byte q + 128, and 0x6400 | byte is 1024 + byte exactly.
template <bool BIAS>
__device__ __forceinline__ f16x8_t codes8(uint32_t lo, uint32_t hi) {
  u32x4_t o;
  lo ^= 0x80808080u;
  hi ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (a bit cast of a vector's element would read its first one: scalars)
    uint32_t two = __builtin_amdgcn_perm(0x64646464u, i < 2 ? lo : hi, (i & 1) ? 0x04030402u : 0x04010400u);
    if constexpr (!BIAS) {
      const f16x2_t c = {(_Float16)1152.0f, (_Float16)1152.0f};
      const f16x2_t v = __builtin_bit_cast(f16x2_t, two) - c;
      two = __builtin_bit_cast(uint32_t, v);
    }
    o[i] = two;
  }
  return __builtin_bit_cast(f16x8_t, o);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  f16x2_t v;
  v[0] = (_Float16)lo;
  v[1] = (_Float16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

// Wave-uniform words through scalar loads (a store or an atomic in the kernel
// keeps the compiler from choosing them by itself; as vector loads they would
// queue behind a page's 16 KB and everything that needs them with it).
typedef const __attribute__((address_space(4))) int32_t* const_i32;
typedef const __attribute__((address_space(4))) float* const_f32;

constexpr float kNegInf = -__builtin_inff(), kMaxF32 = 0x1.fffffep127f;
constexpr int kMaxSplits = 256;   // a lane per split in the join
// Waves of a workgroup, one page each at a time.  Eight instead of four halve
// the partial results of a split, but fewer workgroups fit a CU (48 sequences of
// 0..4095 tokens, 32 / 8 heads of 128: 48 us against 57 at 3 splits; 131071
// tokens on one head: 19.6 against 19.9 at 256).
constexpr int kWaves = 4;

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

// The largest of the wave's numbers, none of them negative.
__device__ __forceinline__ int wave_top(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// The last page worth reading for rows that end before token `end`.  Beyond the
// table: a page that is not there for every row that sees such a token, which is
// the first one past the table or the first one of the row's window.
__device__ __forceinline__ int last_page(const AttnArgs& a, int end) {
  const int start = a.window > 0 ? max(0, end - a.window) / kPage : 0;   // of the last row's window
  return min((end - 1) / kPage, max((int)a.c.width, start));
}

// Pages that the n rows of a sequence of len tokens see: their number, and the first.
__device__ __forceinline__ int pages_of(const AttnArgs& a, int len, int64_t n, int& first) {
  first = 0;
  if (len <= 0 || n <= 0) return 0;
  if (a.window > 0) {
    const int64_t beg = len - n - a.window + 1;
    first = beg > 0 ? (int)(beg / kPage) : 0;
  }
  return last_page(a, len) - first + 1;
}

// The sequence b that slot j works for, its share k of n and the pages it has.
// Every wave works it out from the lengths alone: pages per slot C so that
// sum ceil(pages / C) fits the slots, slots in order of the sequences.  Lane l
// looks at the sequences per * l, ...  False: no work for the slot.
__device__ __forceinline__ bool attn_plan(const AttnArgs& a, int j, bool tell, int& b, int& k, int& n, int& len) {
  constexpr int kMost = 1 << 14;   // (a sum of such stays in range; longer is split in kMaxSplits anyway)
  const int lane = threadIdx.x & 63, nb = a.c.b, per = (nb + 63) >> 6, mine = lane * per;
  auto pages = [&](int s, int tokens) {
    int64_t r0, rows;
    int first;
    kv8_rows(a.c.cu, a.c.rows, nb, s, r0, rows);
    return min(pages_of(a, tokens, rows, first), kMost);
  };
  auto more = [&](int u) { return mine + u < nb ? pages(mine + u, a.c.lens[mine + u]) : 0; };
  auto parts = [](int p, int c) { return min((int)((uint32_t)(p + c - 1) / (uint32_t)c), kMaxSplits); };
  const int len0 = mine < nb ? a.c.lens[mine] : 0, p0 = mine < nb ? pages(mine, len0) : 0;
  int sum = p0, most = p0;
  for (int u = 1; u < per; ++u) {
    const int p = more(u);
    sum += p;
    most = max(most, p);
  }
  most = wave_top(most);
  const int total = __builtin_amdgcn_readlane(wave_scan(sum), 63);
  const int busy = min(nb, per * (int)__popcll(__ballot(sum > 0)));
  // each sequence leaves half a C of its last slot unused
  const int room = a.slots - (busy >> 1);
  int c = max(kWaves, (total + room - 1) / room), cnt, incl;
  // Lengths within an eighth of the longest: the even split, with fewer parts to join
  // (32 sequences of 4096 tokens: 48 us against 52).
  if ((int64_t)most * busy * 7 <= (int64_t)total * 8) c = max(c, (most + a.even - 1) / a.even);
  while (true) {
    cnt = parts(p0, c);
    for (int u = 1; u < per; ++u) cnt += parts(more(u), c);
    incl = wave_scan(cnt);
    if (__builtin_amdgcn_readlane(incl, 63) <= a.slots) break;   // at the latest when c is the longest: slots >= b
    c += 1 + (c >> 4);
  }
  if (tell) {
    int at = incl - cnt;
    for (int u = 0; u < per && mine + u < nb; ++u) {
      const int parts_u = parts(u == 0 ? p0 : more(u), c);
      a.plan[2 * (mine + u)] = at;
      a.plan[2 * (mine + u) + 1] = parts_u;
      at += parts_u;
    }
  }
  const uint64_t mask = __ballot(incl > j);
  if (mask == 0) return false;
  const int at = __builtin_ctzll(mask);
  int base = __builtin_amdgcn_readlane(incl - cnt, at);
  b = at * per;
  len = __builtin_amdgcn_readlane(len0, at);
  n = parts(__builtin_amdgcn_readlane(p0, at), c);
  while (j >= base + n) {          // within the lane's sequences, which hold slot j
    base += n;
    len = ((const_i32)a.c.lens)[++b];
    n = parts(pages(b, len), c);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  n = __builtin_amdgcn_readfirstlane(n);
  k = __builtin_amdgcn_readfirstlane(j - base);
  return true;
}

// SHARED: a.slots > 0.  ROWS: each wave takes a row tile of its own through all
// pages, and row_tiles counts fours of them (one split).
template <int D, int NT, bool SHARED, bool ROWS>
__global__ __launch_bounds__(64 * kWaves) void attn_kv8_kernel(AttnArgs a) {
  constexpr int KC = D / 64;        // 64-channel chunks of a key
  constexpr int DT = D / 16;        // 16-channel tiles of a value
  constexpr bool kEarlyV = D <= 192 && D * NT <= 256;   // values in flight with the keys, where registers allow
  __shared__ float sm_m[ROWS ? 1 : kWaves][16 * NT], sm_l[ROWS ? 1 : kWaves][16 * NT];
  __shared__ f32x4_t sm_o[ROWS ? 1 : kWaves][DT][64];
  const int lane = threadIdx.x & 63, i = lane & 15, qd = lane >> 4;
  const int wave = wave_id_uniform();
  // Splits slowest: workgroups go to the 8 XCDs in turn, and the late splits
  // of short sequences, which are empty, must not all fall to the same ones.
  const int h = blockIdx.x / a.row_tiles, rt = ROWS ? blockIdx.x % a.row_tiles * kWaves + wave : blockIdx.x % a.row_tiles;
  int b = blockIdx.y, split = blockIdx.z, splits = a.splits, len;
  if constexpr (SHARED) {
    const bool tell = blockIdx.x == 0 && blockIdx.y == 0 && wave == 0;
    if (!attn_plan(a, blockIdx.y, tell, b, split, splits, len)) return;
  }
  const const_i32 trow = (const_i32)(a.c.table + (size_t)b * a.c.width);
  const int width = (int)a.c.width;
  // Without a window the first page does not depend on the length: its table
  // entry is on its way together with the length.
  const int guess = SHARED || ROWS ? 0 : (int)min((int64_t)split * a.chunk + wave, (int64_t)width - 1);
  const int guessed = trow[guess];
  if constexpr (!SHARED) len = ((const_i32)a.c.lens)[b];
  len = max(len, 0);
  int64_t r0, n64;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, n64);
  const int nq = (int)(n64 < a.max_q ? n64 : a.max_q);
  const int nrows = nq * a.group;
  const int row0 = rt * 16 * NT;
  if (row0 >= nrows) return;
  // The last query row is the sequence's last token.
  const int shift = len - (int)n64;                  // position of query row t: shift + t
  const int t_lo = group_of(a, row0), t_hi = group_of(a, min(row0 + 16 * NT - 1, nrows - 1));
  const int pos_hi = shift + t_hi, pos_lo = shift + t_lo;
  const int tok_end = pos_hi + 1;                    // tokens [tok_beg, tok_end) are seen by some row
  const int tok_beg = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
  int p_beg = 0, p_end = 0;
  if (tok_end > tok_beg) {
    const int first = tok_beg / kPage;
    const int last = last_page(a, tok_end);
    if constexpr (SHARED) {
      // even shares of the pages that the whole sequence sees
      int from;
      const int all = pages_of(a, len, n64, from), share = all / splits, more = all % splits;
      const int beg = from + split * share + min(split, more);
      p_beg = max(beg, first);
      p_end = split + 1 < splits ? min(beg + share + (split < more ? 1 : 0), last + 1) : last + 1;
    } else {
      // `chunk` pages a split, the last one what is left: equal work for every
      // workgroup whatever the lengths
      p_beg = (int)min(first + (int64_t)split * a.chunk, (int64_t)last + 1);
      p_end = split + 1 < splits ? (int)min((int64_t)p_beg + a.chunk, (int64_t)last + 1) : last + 1;
    }
  }
  // row t of the partial results
  const size_t part0 = SHARED ? (size_t)blockIdx.y * a.max_q : (size_t)split * a.c.rows + r0;

  if (p_beg >= p_end && splits > 1) {                // nothing here: say so to the join, and no more
    const int r = row0 + (int)threadIdx.x;
    if ((int)threadIdx.x < 16 * NT && r < nrows) {
      const int t = group_of(a, r), g = r - t * a.group;
      float* const ml = a.part_ml + ((part0 + t) * a.hq + h * a.group + g) * 2;
      ml[0] = kNegInf;
      ml[1] = 0.0f;
    }
    return;
  }

  const bool alone = !ROWS && p_end - p_beg <= 1;    // one wave has the only page
  const int first_page = p_beg + (ROWS ? 0 : wave);
  constexpr int kStep = ROWS ? 1 : kWaves;

  // Rows of this lane, as fp16 q 2^(8 - e) with 2^e just above the row's
  // largest channel: exact but for channels 2^-21 of that one.  The keys'
  // bias of 1152 comes off in the accumulator's first value.
  int pos[NT];
  float rscale[NT], corr[NT];
  f16x8_t qf[NT][2 * KC];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 16 * n + i;
    const bool on = r < nrows && (!alone || wave == 0);
    const int t = group_of(a, r), g = r - t * a.group;
    pos[n] = on ? shift + t : -1;
    const uint16_t* src = a.q + (r0 + t) * a.q_ts + (int64_t)(h * a.group + g) * a.q_hs + 16 * qd;
    u32x4_t raw[2 * KC];
    float mx = 0.0f;
#pragma unroll
    for (int c = 0; c < 2 * KC; ++c) {
      raw[c] = u32x4_t{0u, 0u, 0u, 0u};
      if (on) raw[c] = *reinterpret_cast<const u32x4_t*>(src + 64 * (c >> 1) + 8 * (c & 1));
    }
#pragma unroll
    for (int c = 0; c < 2 * KC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(raw[c][e] << 16)), fabsf(__uint_as_float(raw[c][e] & 0xffff0000u))));
    mx = fold_quads(mx, [](float x, float y) { return fmaxf(x, y); });
    const int ex = mx > 0.0f && mx < __builtin_inff() ? __builtin_amdgcn_frexp_expf(mx) : 8;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 2 * KC; ++c) {
      u32x4_t o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = pack_f16(__builtin_ldexpf(__uint_as_float(raw[c][e] << 16), 8 - ex),
                                      __builtin_ldexpf(__uint_as_float(raw[c][e] & 0xffff0000u), 8 - ex));
        const f16x2_t v = __builtin_bit_cast(f16x2_t, two);
        sum += (float)v[0] + (float)v[1];
        o[e] = two;
      }
      qf[n][c] = __builtin_bit_cast(f16x8_t, o);
    }
    corr[n] = -1152.0f * fold_quads(sum, [](float x, float y) { return x + y; });
    rscale[n] = __builtin_ldexpf(a.scale_log2, ex - 8);
  }

  float m[NT], l[NT];
  float pe[NT], pmul[NT];           // a whole number, p * vs < 2^(pe + 1) so far, and 2^(kTopExp - pe): o holds O * pmul
  f32x4_t o[NT][DT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
    pe[n] = kMinExp;
    pmul[n] = __builtin_ldexpf(1.0f, kTopExp - kMinExp);
#pragma unroll
    for (int t = 0; t < DT; ++t) o[n][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto entry = [&](int p) {         // the page, or -1
    const int e = p == guess ? guessed : p < width ? trow[p] : -1;
    return p < width && e >= 0 && e < a.c.pages ? e : -1;
  };
  bool missing = false;
  int next = first_page < p_end ? entry(first_page) : 0;
  for (int p = first_page; p < p_end; p += kStep) {
    const int page = next;
    const int held = page < 0 ? 0 : page;            // reads stay inside; its scales become NaN below
    const int8_t* const kc = a.c.codes + kv8_base(held, a.c.hkv, h, D);
    const const_f32 sc = (const_f32)(a.c.scales + ((size_t)held * a.c.hkv + h) * 8);
    u32x4_t kr[4][KC], vr[DT];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk)
#pragma unroll
      for (int c = 0; c < KC; ++c)
        kr[blk][c] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(kc + (16 * blk + i) * D + 64 * c + 16 * qd));
    auto load_v = [&] {
#pragma unroll
      for (int t = 0; t < DT; ++t)
        vr[t] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(kc + kPage * D + 1024 * t + 64 * i + 16 * qd));
    };
    if constexpr (kEarlyV) load_v();
    float ks[4], vs[4];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
      ks[blk] = sc[blk];
      vs[blk] = sc[4 + blk];
    }
    if (p + kStep < p_end) next = entry(p + kStep);
    missing |= page < 0;
    const int j0 = p * kPage;
    const bool edge = j0 + kPage - 1 > pos_lo || (a.window > 0 && j0 <= pos_hi - a.window);   // uniform

    f32x4_t s[NT][4];
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][blk] = f32x4_t{corr[n], corr[n], corr[n], corr[n]};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const f16x8_t k0 = codes8<true>(kr[blk][c][0], kr[blk][c][1]), k1 = codes8<true>(kr[blk][c][2], kr[blk][c][3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][2 * c], s[n][blk], 0, 0, 0);
          s[n][blk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][2 * c + 1], s[n][blk], 0, 0, 0);
        }
      }
    }
    if constexpr (!kEarlyV) load_v();

    // The exponents of the value scales (uniform).  A scale that is infinite or NaN and
    // a page that is not there turn the scores into NaN, which reaches the rows that see it.
    int vexp[4], vtop = kMinExp;
#pragma unroll
    for (int blk = 0; blk < 4; ++blk) {
      const int ex = (int)(__float_as_uint(vs[blk]) >> 23 & 0xff);
      vexp[blk] = ex < 255 ? max(ex - 127, kMinExp) : kMinExp;
      vtop = max(vtop, vexp[blk]);
      const bool bad = page < 0 || ex == 255 || (__float_as_uint(ks[blk]) >> 23 & 0xff) == 255;
      if (bad) ks[blk] = __uint_as_float(0x7fc00000u);
    }

    f16x8_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top[4];                 // of the lane's scores in a block
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) {
        const float f = ks[blk] * rscale[n];
        top[blk] = kNegInf;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = s[n][blk][e] * f;
          if (edge) {
            const int j = j0 + 16 * blk + 4 * qd + e;
            v = j <= pos[n] && (a.window <= 0 || j > pos[n] - a.window) ? v : kNegInf;
          }
          s[n][blk][e] = v;
          top[blk] = fmaxf(top[blk], v);
        }
      }
      auto larger = [](float x, float y) { return fmaxf(x, y); };
      const float mx = fold_quads(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), larger);
      const float m_new = fmaxf(m[n], ceilf(mx));
      const float base = m_new == kNegInf ? 0.0f : m_new;   // nothing seen yet: every p is 0
      const float pe_old = pe[n] + (m[n] - base);           // relative to the new maximum
      // Nothing to do while no maximum moved and the page's largest p with its largest
      // scale stays below what the row has seen; else the largest p * vs counts, from
      // the largest p of each block.
      if (__ballot(m_new > m[n] || mx - base + (float)vtop > pe_old) != 0) {
        float ptop = kNegInf;
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) ptop = fmaxf(ptop, top[blk] - base + (float)vexp[blk]);
        const float pe_new = fmaxf(fmaxf(pe_old, ceilf(fold_quads(ptop, larger))), (float)kMinExp);
        const float f = __builtin_amdgcn_exp2f(pe_old - pe_new);
        l[n] *= __builtin_amdgcn_exp2f(m[n] - base);
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][t][e] *= f;
        m[n] = m_new;
        pe[n] = pe_new;
        pmul[n] = __builtin_ldexpf(1.0f, kTopExp - (int)pe_new);
      }
      // Scales as the operands want them, finite so that a p of 0 stays 0: the bound only
      // counts beside a scale that is 2^112 smaller, where p is below 2^-113, and for the
      // blocks that are NaN or that the row does not see.
      float vn[4];
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) vn[blk] = __builtin_amdgcn_fmed3f(vs[blk] * pmul[n], -kMaxF32, kMaxF32);
      u32x4_t w[2];
      float sum = 0.0f;
#pragma unroll
      for (int blk = 0; blk < 4; ++blk) {
        float pv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[n][blk][e] - base);
          sum += x;
          pv[e] = x * vn[blk];
        }
        w[blk >> 1][2 * (blk & 1)] = pack_f16(pv[0], pv[1]);
        w[blk >> 1][2 * (blk & 1) + 1] = pack_f16(pv[2], pv[3]);
      }
      l[n] += sum;
      pf[n][0] = __builtin_bit_cast(f16x8_t, w[0]);
      pf[n][1] = __builtin_bit_cast(f16x8_t, w[1]);
    }
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      const f16x8_t v0 = codes8<false>(vr[t][0], vr[t][1]), v1 = codes8<false>(vr[t][2], vr[t][3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[n][0], o[n][t], 0, 0, 0);
        o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[n][1], o[n][t], 0, 0, 0);
      }
    }
  }
  if (missing && a.status && lane == 0) atomicOr(a.status, QG_FLAG_PAGE);
  float vback[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) vback[n] = __builtin_ldexpf(1.0f, (int)pe[n] - kTopExp);

  auto store = [&](int64_t row, int d, const f32x4_t& v, float ll) {   // O / l of the output's row
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    const f32x4_t y{v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    if (a.out_f32)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (size_t)row * D + d) = y;
    else
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + (size_t)row * D + d) =
          u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
  };
  if constexpr (ROWS) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] = fold_quads(l[n], [](float x, float y) { return x + y; });
      const int r = row0 + 16 * n + i;
      if (r >= nrows) continue;
      const int t = group_of(a, r), g = r - t * a.group;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        store((r0 + t) * a.hq + h * a.group + g, 16 * dt + 4 * qd,
              f32x4_t{o[n][dt][0] * vback[n], o[n][dt][1] * vback[n], o[n][dt][2] * vback[n], o[n][dt][3] * vback[n]}, l[n]);
    }
    return;
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
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm_m[w][16 * n + i]);
    const float base = mm == kNegInf ? 0.0f : mm;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) ll += sm_l[w][16 * n + i] * __builtin_amdgcn_exp2f(sm_m[w][16 * n + i] - base);
    const float f = __builtin_amdgcn_exp2f(m[n] - base) * vback[n];
    if (n > 0) __syncthreads();
    if (!alone || wave == 0)
#pragma unroll
      for (int t = 0; t < DT; ++t)
        sm_o[wave][t][lane] = f32x4_t{o[n][t][0] * f, o[n][t][1] * f, o[n][t][2] * f, o[n][t][3] * f};
    __syncthreads();
    const int r = row0 + 16 * n + i;
    const int t = group_of(a, r), g = r - t * a.group;
    const int64_t row = (r0 + t) * a.hq + h * a.group + g;     // row of the output
    const size_t prow = (part0 + t) * a.hq + h * a.group + g;
    const bool on = r < nrows;
    for (int dt = wave; dt < DT; dt += kWaves) {
      f32x4_t v = sm_o[0][dt][lane];
      if (!alone)
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
          const f32x4_t u = sm_o[w][dt][lane];
          v = f32x4_t{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
        }
      if (!on) continue;
      const int d = 16 * dt + 4 * qd;
      if (splits > 1) {
        if (mm != kNegInf || ll != 0.0f)
          *reinterpret_cast<f32x4_t*>(a.part_o + prow * D + d) = v;
      } else {
        store(row, d, v, ll);
      }
    }
    if (splits > 1 && on && wave == 0 && qd == 0) {
      float* const ml = a.part_ml + prow * 2;
      ml[0] = mm;
      ml[1] = ll;
    }
  }
}

// Where the partial results of a row are: split s of head hd in row at(s, hd).
struct JoinParts {
  int n, hq;
  size_t first, step;
  __device__ __forceinline__ size_t at(int s, int hd) const { return (first + s * step) * hq + hd; }
};
template <bool SHARED>
__device__ __forceinline__ JoinParts join_parts(const AttnArgs& a, int b, int64_t row, int t) {
  if constexpr (SHARED) {
    const const_i32 plan = (const_i32)(a.plan + 2 * (size_t)b);
    return {plan[1], a.hq, (size_t)plan[0] * a.max_q + t, (size_t)a.max_q};
  } else {
    return {a.splits, a.hq, (size_t)row, (size_t)a.c.rows};
  }
}

// The splits of one row and head, joined in a fixed order: the factors
// 2^(m_s - M) first (a lane per split), then O.  A workgroup takes 32 channels,
// 32 groups of 8 lanes taking splits in turn, so that with many splits all
// their loads are in flight at once.  Splits that saw nothing wrote no O and
// are not read.
template <int D, bool SHARED>
__global__ __launch_bounds__(256) void attn_kv8_join_kernel(AttnArgs a) {
  __shared__ float sm_f[kMaxSplits], sm_w[4], sm_l[4];
  __shared__ f32x4_t sm_o[32][8];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform();
  const int b = blockIdx.z, t = blockIdx.y, hd = blockIdx.x / (D / 32), d0 = blockIdx.x % (D / 32) * 32;
  int64_t r0, n;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, n);
  if (t >= n) return;
  const JoinParts parts = join_parts<SHARED>(a, b, r0 + t, t);
  if (SHARED && parts.n == 1) return;
  const size_t row = (size_t)(r0 + t) * a.hq + hd;
  float m = kNegInf, l = 0.0f;
  if (tid < parts.n) {
    const float* const ml = a.part_ml + parts.at(tid, hd) * 2;
    m = ml[0];
    l = ml[1];
  }
  float mm = m;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) mm = fmaxf(mm, __shfl_xor(mm, o));
  if (lane == 0) sm_w[wave] = mm;
  __syncthreads();
  mm = fmaxf(fmaxf(sm_w[0], sm_w[1]), fmaxf(sm_w[2], sm_w[3]));
  const float f = mm == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - mm);
  float ll = mm == kNegInf ? l : l * f;      // nothing seen: l is 0, or NaN
#pragma unroll
  for (int o = 1; o < 64; o *= 2) ll += __shfl_xor(ll, o);
  if (lane == 0) sm_l[wave] = ll;
  sm_f[tid] = f;
  __syncthreads();
  ll = (sm_l[0] + sm_l[1]) + (sm_l[2] + sm_l[3]);
  const int g = tid >> 3, c = tid & 7;
  f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* const po = a.part_o + d0 + 4 * c;
#pragma unroll
  for (int u = 0; u < kMaxSplits / 32; ++u) {
    const int s = g + 32 * u;
    const float w = sm_f[s];
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (s < parts.n && w != 0.0f) x = *reinterpret_cast<const f32x4_t*>(po + parts.at(s, hd) * D);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(w, x[e], v[e]);
  }
  sm_o[g][c] = v;
  __syncthreads();
  if (tid >= 32) return;
  float y = 0.0f;
#pragma unroll
  for (int u = 0; u < 32; ++u) y += sm_o[u][tid >> 2][tid & 3];
  y *= ll == 0.0f ? 0.0f : 1.0f / ll;
  const size_t at = row * D + d0 + tid;
  if (a.out_f32)
    static_cast<float*>(a.out)[at] = y;
  else
    static_cast<uint16_t*>(a.out)[at] = (uint16_t)f32_to_bf16_rne(y);
}

// The same for few splits: a lane takes 4 channels of a row through all of
// them, 16 at a time, a workgroup 256 / (D / 4) heads.
typedef float f32x2_t __attribute__((ext_vector_type(2)));
constexpr int kFewSplits = 16;
constexpr int64_t kJoinWide = 2 * kCUs;        // workgroups of the other join
template <int D, bool SHARED>
__global__ __launch_bounds__(256) void attn_kv8_join_few_kernel(AttnArgs a) {
  constexpr int C = D / 4, R = 256 / C;
  const int g = threadIdx.x / C, c = threadIdx.x % C;
  const int b = blockIdx.z, t = blockIdx.y, hd = blockIdx.x * R + g;
  int64_t r0, rows;
  kv8_rows(a.c.cu, a.c.rows, a.c.b, b, r0, rows);
  if (t >= rows) return;
  const JoinParts parts = join_parts<SHARED>(a, b, r0 + t, t);
  if (SHARED && parts.n == 1) return;          // written by the workgroup that did it all
  if (g >= R || hd >= a.hq) return;
  const size_t row = (size_t)(r0 + t) * a.hq + hd;
  float mm = kNegInf, ll = 0.0f;
  f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < parts.n; s0 += kFewSplits) {
    f32x2_t ml[kFewSplits];
    float top = mm;
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) {
      ml[s] = f32x2_t{kNegInf, 0.0f};
      if (s0 + s < parts.n) ml[s] = *reinterpret_cast<const f32x2_t*>(a.part_ml + parts.at(s0 + s, hd) * 2);
    }
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) top = fmaxf(top, ml[s][0]);
    const float base = top == kNegInf ? 0.0f : top, back = __builtin_amdgcn_exp2f(mm - base);
    ll *= back;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= back;
#pragma unroll
    for (int s = 0; s < kFewSplits; ++s) {
      const float f = __builtin_amdgcn_exp2f(ml[s][0] - base);
      ll += ml[s][1] * f;                      // (nothing seen: 0, or NaN)
      f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
      if (s0 + s < parts.n && f != 0.0f)
        x = *reinterpret_cast<const f32x4_t*>(a.part_o + parts.at(s0 + s, hd) * D + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(f, x[e], y[e]);
    }
    mm = top;
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  if (a.out_f32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + row * D + 4 * c) = y;
  else
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + row * D + 4 * c) =
        u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

// Row tiles a wave takes at once: two where a head has more than 16 rows, so
// that a page's codes are converted once for both (8 sequences of 8192 tokens, 3
// rows on 64 / 8 heads of 128: 35 us against 53; of 256: 75 against 104).
int attn_kv8_nt(int64_t rows_per_head) { return rows_per_head > 16 ? 2 : 1; }

// Pages that a sequence's rows can see.
static int64_t seen_pages(int64_t max_len, int window, int64_t max_q) {
  int64_t seen = max_len;
  if (window > 0 && window + max_q + kPage < seen) seen = window + max_q + kPage;
  return (seen + kPage - 1) / kPage;
}

// Workgroups that a CU holds at once, by their registers.
static int resident(int d, int nt) { return d * nt <= 64 ? 4 : d * nt <= 128 ? 3 : d * nt <= 256 ? 2 : 1; }

// Splits of a sequence's pages over workgroups, by what a split costs: rounds of a
// page per wave, of `lat` each when nothing else limits them (page and arithmetic,
// measured on few workgroups), or the pages of the fullest CU at its share of the
// bandwidth, 25 bytes a ns; 3 us for the join.  Tried are the splits that fill
// the CUs once, twice, ... up to what they hold, each also with whole rounds.
// Against the best of 11 splits from 1 to 36 at 96 shapes (64, 128 and 256 channels, 1
// to 16 sequences of 300 to 9000 tokens, 1 and 4 rows) the choice costs 2.4 % on
// average and 11 % at most; two workgroups per CU throughout cost up to 54 % (2 x 4
// rows of 64 / 8 heads of 256, 9000 tokens: 49 us, now 32).
static int attn_splits(int64_t b, int hkv, int d, int64_t rows_per_head, int64_t max_len, int window, int64_t max_q) {
  const int nt = attn_kv8_nt(rows_per_head), held = resident(d, nt);
  const int64_t units = b * hkv * ((rows_per_head + 16 * nt - 1) / (16 * nt));
  const int64_t pages = seen_pages(max_len, window, max_q);
  // A page for every wave; of 256 channels for every second one, which alone get
  // their pages sooner (1 sequence of 1000 tokens on 8 heads: 12.2 us against 13.6).
  const int64_t least_pages = d > 192 ? 2 : kWaves;
  if (pages <= least_pages || units >= held * kCUs) return 1;
  const int64_t joined = b * hkv * rows_per_head * (d / 32);
  // tenths of a us
  const int64_t lat = (nt == 1 ? 7 : 13) + d / 9, page = d / 20;
  auto rounds_of = [&](int64_t s) { return ((pages + s - 1) / s + kWaves - 1) / kWaves; };
  auto cost = [&](int64_t s) {
    const int64_t full = (units * s + kCUs - 1) / kCUs, turns = (full + held - 1) / held, rounds = rounds_of(s);
    const bool pair = d > 192 && (pages + s - 1) / s <= 2;
    const int64_t alone = rounds * lat * (pair ? 7 : 10) / 10;
    const int64_t shared = std::min<int64_t>(full, held) * (pair ? 2 : rounds * kWaves) * page;
    const int64_t join = s == 1 ? 0 : 30 + (s > kFewSplits ? (joined > kJoinWide ? (s - 1) / kFewSplits * 20 : 5) : 0);
    return turns * std::max(alone, shared) + (turns - 1) * 40 + join;
  };
  int64_t best = 1, least = cost(1);
  auto take = [&](int64_t s) {
    s = std::min<int64_t>({s, (pages + least_pages - 1) / least_pages, kMaxSplits});
    if (s <= 1) return;
    const int64_t c = cost(s);
    if (c <= least) best = s, least = c;
  };
  for (int c = 1; c <= held; ++c) {
    const int64_t s = c * kCUs / units;
    if (s < 1) continue;
    const int64_t r = rounds_of(s);
    take(s);
    take((pages + kWaves * r - 1) / (kWaves * r));
    if (r > 1) take((pages + kWaves * (r - 1) - 1) / (kWaves * (r - 1)));
  }
  return (int)best;
}

// How a call's pages are split: each sequence's in `splits`, or, where slots > 0,
// over `slots` workgroups per head and row tile by the sequences' lengths, which
// only the GPU knows.  Sharing out is for splits of many pages: a workgroup finds
// its sequence first (about 1 us), and equal splits of up to five pages a wave
// leave little to gain (1 sequence of 60000 tokens and 31 of 100..600, 32 / 8
// heads of 128: 40 us against 416; 48 of 10..4095 in any order: 45 against 60;
// 16 of 10..8192 on 64 / 8: 31 against 42).  Sequences of about one length get the even
// split all the same: 32 of 4096 take 48 us with the preparation and a join that finds
// nothing, against 46 for one split from the start, which 32 of 10..4096 pay with 38
// against 34.
// As many slots as workgroups are resident at once: with 2 a CU instead of 3 the
// 48 take 52 us, with 4 they take 47.
AttnSplit attn_kv8_split(int64_t b, int64_t rows, int hkv, int d, int64_t rows_per_head, int64_t max_len, int window,
                         int64_t max_q) {
  const int s = attn_splits(b, hkv, d, rows_per_head, max_len, window, max_q);
  const int nt = attn_kv8_nt(rows_per_head);
  const int64_t units = hkv * ((rows_per_head + 16 * nt - 1) / (16 * nt));
  const int64_t slots = std::max((resident(d, nt) * kCUs + units - 1) / units, b + b / 2);
  // (four times the row tiles that fill the card: 16 sequences of 3000 tokens, 64 rows on
  // 64 / 8 heads of 128, 226 us with a row tile a wave against 280)
  if (units * b >= 4 * resident(d, nt) * kCUs && rows_per_head > 16 * nt) return {1, 0};
  if (max_q * b > 2 * rows || seen_pages(max_len, window, max_q) <= 5 * kWaves * s || slots > 65535)
    return {s, 0};
  return {s, (int)slots};
}

template <int D, int NT, bool SHARED, bool ROWS = false>
static hipError_t launch_attn_t(const AttnArgs& a, hipStream_t stream) {
  const int x = a.row_tiles * a.c.hkv;
  const dim3 grid = SHARED ? dim3(x, a.slots) : dim3(x, a.c.b, a.splits);
  hipLaunchKernelGGL((attn_kv8_kernel<D, NT, SHARED, ROWS>), grid, dim3(64 * kWaves), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!SHARED && a.splits == 1)) return e;
  // Many splits of few rows: a workgroup for 32 channels of a row; with many rows
  // the other, 16 splits at a time (36 splits of 2 x 4 rows of 64 heads of 128, 9000
  // tokens: 26.7 us in all against 28.0 that way).
  constexpr int R = 256 / (D / 4);
  const bool few = SHARED ? a.slots <= kFewSplits * a.c.b : a.splits <= kFewSplits;
  if (few || (int64_t)a.hq * (D / 32) * a.max_q * a.c.b > kJoinWide)
    hipLaunchKernelGGL((attn_kv8_join_few_kernel<D, SHARED>), dim3((a.hq + R - 1) / R, a.max_q, a.c.b), dim3(256), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((attn_kv8_join_kernel<D, SHARED>), dim3(a.hq * (D / 32), a.max_q, a.c.b), dim3(256), 0, stream,
                       a);
  return hipGetLastError();
}

hipError_t launch_attn_kv8(const Kv8Args& c, const void* q, int64_t q_ts, int64_t q_hs, int hq, int max_q,
                           int64_t max_len, int window, float scale, void* out, int out_f32, AttnSplit by, float* part,
                           uint32_t* status, hipStream_t stream) {
  const int group = hq / c.hkv;
  const int64_t rows_per_head = (int64_t)max_q * group;
  const int nt = attn_kv8_nt(rows_per_head);
  const int64_t pages = seen_pages(max_len, window, max_q);
  const int splits = by.slots > 0 ? 1 : by.splits;
  const int chunk = pages > splits ? (int)((pages + splits - 1) / splits) : 1;
  AttnArgs a{c, static_cast<const uint16_t*>(q), q_ts, q_hs, hq, group, max_q, window, splits, chunk,
             (int)((rows_per_head + 16 * nt - 1) / (16 * nt)), group > 1 ? (uint32_t)(((uint64_t)1 << 32) / group) : 0u,
             scale * 1.44269504088896340736f, out, out_f32,
             part, nullptr, by.slots, by.splits, nullptr, status};
  if (part) {
    const size_t partial = (by.slots > 0 ? (size_t)by.slots * max_q : (size_t)splits * c.rows) * hq;
    a.part_ml = part + partial * c.d;
    a.plan = reinterpret_cast<int32_t*>(a.part_ml + partial * 2);
  }
  // A row tile a wave instead of a page a wave: where there is hardly a second page,
  // and where the row tiles fill the card one and a half times, there is nothing to
  // join then and no wave waits (57 sequences of 17..45 tokens, 37 rows on 20 / 4 heads of 256: 30 us
  // against 71; 16 of 1000, 64 on 64 / 8 of 128: 86 against 106; at half as many row
  // tiles, 2 of 256: 17 against 11).  One tile at a time for up to two pages (12
  // of 64, 61 on 40 / 8 of 64: 6.8 against 8.6), two above (86 against 134).
  const int64_t units = (int64_t)a.row_tiles * c.hkv * c.b;
  const bool rows = splits == 1 && by.slots == 0 && a.row_tiles > 1 &&
                    (pages <= 2 || 2 * units >= 3 * resident(c.d, nt) * kCUs);
  const int tall = rows && pages <= 2 ? 1 : nt;
  if (rows) a.row_tiles = (int)((rows_per_head + 16 * tall * kWaves - 1) / (16 * tall * kWaves));
  switch (c.d * 4 + tall) {
#define QG_ATTN(D, NT) \
  case D * 4 + NT:          \
    if (rows) return launch_attn_t<D, NT, false, true>(a, stream);                                          \
    return by.slots > 0 ? launch_attn_t<D, NT, true>(a, stream) : launch_attn_t<D, NT, false>(a, stream);
    QG_ATTN(64, 1) QG_ATTN(64, 2) QG_ATTN(128, 1) QG_ATTN(128, 2) QG_ATTN(192, 1) QG_ATTN(192, 2)
    QG_ATTN(256, 1) QG_ATTN(256, 2)
#undef QG_ATTN
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qg
