// verify.hip -- drafted tokens against the target's probabilities, and the
// next token (qg_verify_drafts).
//
// A sequence with n drafted tokens has n + 1 rows of the target's probabilities p
// and n of the draft's q.  Draft x of row i is accepted while u q_i(x) < p_i(x); at
// the first that is not, the next token is drawn from max(p - q, 0) of that row,
// after the last one from p: the first j whose running sum exceeds u' times the
// whole sum.  So the tokens are distributed as if the target alone had drawn them.
//
// Sums are in 64 bits: a vocabulary's running sums in 32 would move a border
// between tokens by a ten-thousandth of a likely token's share.  Where running
// sums decide, they are sums of whole numbers (a share of 2^61): exact in any
// order, so a token without a share is never drawn.
//
// Only the one row that counts is read, but for a few values.  It falls into pieces of
// 512 tokens or more, a wave's work: their sums first, then the piece with the
// border in it, read again.
#include "layer_common.h"
#include "w4_common.h"
#include "wave.h"

namespace qg {

constexpr int kPiece = 512;            // tokens, 8 a lane
constexpr int kMaxPieces = 1024;       // a row's, 16 a lane of the wave that draws; longer pieces where it has more
constexpr int kVerifyOnePieces = 256;   // those whose sums one workgroup keeps in LDS

template <bool HALF>
__device__ __forceinline__ float prob(const void* p, size_t at) {
  if constexpr (HALF) return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
  return static_cast<const float*>(p)[at];
}

struct VerifyRow {                     // where the next token of a sequence comes from
  int64_t first, drafts;               // rows of the target: first .. first + drafts
  int accepted;
  size_t p, q;                         // first element of the target's row, and of the draft's
  bool two;                            // there is a draft's row
  int without;                         // the rejected token where drafts are certain, or -1
  bool bad;                            // a drafted token outside the vocabulary
};

// Rows of sequence b; false where its offsets are not in order, or where one of its rows, of
// the target or of the drafts, is not there.
__device__ __forceinline__ bool verify_rows(const VerifyArgs& a, int b, VerifyRow& r) {
  r.bad = false;
  r.first = a.cu[b];
  const int64_t end = a.cu[b + 1];
  r.drafts = end - r.first - 1;
  return r.drafts >= 0 && end <= a.rows && r.first >= b && r.first - b + r.drafts <= a.rows - a.b;
}

// The row behind `accepted` drafts.
__device__ __forceinline__ void verify_at(const VerifyArgs& a, int b, int accepted, VerifyRow& r) {
  r.accepted = accepted;
  const int64_t d = r.first - b + accepted;
  r.p = (size_t)(r.first + accepted) * a.v;
  r.q = (size_t)d * a.v;
  r.two = accepted < r.drafts && a.draft != nullptr;
  r.without = accepted < r.drafts && !a.draft ? __builtin_amdgcn_readfirstlane(a.tokens[d]) : -1;
}

// The first rejected draft of sequence b, by a whole wave.
template <bool HALF>
__device__ __forceinline__ void verify_find(const VerifyArgs& a, int b, VerifyRow& r) {
  const int lane = threadIdx.x & 63;
  int64_t accepted = r.drafts;
  for (int64_t i0 = 0; i0 < r.drafts; i0 += 64) {
    const int64_t i = i0 + lane, d = r.first - b + i;
    bool ok = true, out = false;
    if (i < r.drafts) {
      const int x = a.tokens[d];
      const double u = (double)a.u[d];
      out = x < 0 || x >= a.v;
      ok = false;
      if (!out) {
        const double p = (double)prob<HALF>(a.target, (size_t)(r.first + i) * a.v + x);
        const double q = a.draft ? (double)prob<HALF>(a.draft, (size_t)d * a.v + x) : 1.0;
        ok = u * q < p;
      }
    }
    const uint64_t no = __ballot(!ok);
    if (no != 0) {
      const int at = __builtin_ctzll(no);
      r.bad = (__ballot(out) >> at & 1) != 0;
      accepted = i0 + at;
      break;
    }
  }
  verify_at(a, b, __builtin_amdgcn_readfirstlane((int)accepted), r);
}

// What a token weighs: max(p - q, 0); a NaN counts as 0.
__device__ __forceinline__ double verify_left(float p, float q) {
  return fmax((double)p - (double)q, 0.0);
}

// Eight tokens a lane of the 512 from j0 on: in order (lane l: 8 l ..) or, for
// sums, as they are read best.  Tokens from v on weigh nothing (they are past the
// end of the view), nor does the one that was rejected where drafts are certain.
template <bool HALF, bool ORDER>
struct VerifyEight {
  typedef uint32_t u32x8_t __attribute__((ext_vector_type(8)));
  u32x8_t w = {}, x = {};                // p and q as they lie in memory: pairs of bf16 where `whole`
  __device__ __forceinline__ void load(const VerifyArgs& a, const VerifyRow& r, int64_t j0) {
    constexpr int kSize = HALF ? 2 : 4;
    const int lane = threadIdx.x & 63;
    const int bytes = (int)min((int64_t)kPiece, a.v - j0) * kSize;
    const BufView pv(static_cast<const char*>(a.target) + (r.p + j0) * kSize, bytes);
    const BufView qv(static_cast<const char*>(r.two ? a.draft : a.target) + (r.two ? (r.q + j0) * kSize : 0), r.two ? bytes : 0);
    if (a.whole) {                       // rows start on 16 bytes and end so: 16 bytes are all there or not
#pragma unroll
      for (int h = 0; h < (HALF ? 1 : 2); ++h) {
        const u32x4_t p = pv.b128<false>((HALF ? 16 : 32) * lane + 16 * h), q = qv.b128<false>((HALF ? 16 : 32) * lane + 16 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * h + i] = p[i], x[4 * h + i] = q[i];
      }
    } else {                             // 64 neighbours at a time where the order is free
      const uint32_t at = kSize * (ORDER ? 8 * lane : lane), step = kSize * (ORDER ? 1 : 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = HALF ? pv.b16(at + i * step) : pv.b32(at + i * step);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = HALF ? qv.b16(at + i * step) : qv.b32(at + i * step);
    }
  }
  __device__ __forceinline__ void values(const VerifyArgs& a, const VerifyRow& r, int64_t j0, float (&p)[8], float (&q)[8]) const {
    const int lane = threadIdx.x & 63;
    const bool order = ORDER || a.whole;
    // (bf16 in pairs are taken apart here: w[4 ..] is not loaded then)
    const bool pairs = HALF && a.whole;
    const uint32_t odd = 0xffff0000u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0 = w[2 * i], w1 = w[2 * i + 1], x0 = x[2 * i], x1 = x[2 * i + 1];
      if constexpr (HALF) w0 <<= 16, w1 <<= 16, x0 <<= 16, x1 <<= 16;
      if (pairs) w0 = w[i] << 16, w1 = w[i] & odd, x0 = x[i] << 16, x1 = x[i] & odd;
      p[2 * i] = __uint_as_float(w0), p[2 * i + 1] = __uint_as_float(w1);
      q[2 * i] = __uint_as_float(x0), q[2 * i + 1] = __uint_as_float(x1);
    }
    if (r.without >= j0 && r.without < j0 + kPiece) {
      const int not_it = (int)(r.without - j0);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((order ? 8 * lane + i : 64 * i + lane) == not_it) p[i] = 0.0f;
    }
  }
};

// The sums of the pieces first, first + step, ... below a.pieces, each given to
// take(piece, sum); the loads of the next 512 tokens are in flight while these are added.
template <bool HALF, class Take>
__device__ __forceinline__ void verify_sums(const VerifyArgs& a, const VerifyRow& r, int first, int step, Take take) {
  if (first >= a.pieces) return;
  VerifyEight<HALF, false> now, next;
  int64_t j0 = first * a.piece;
  now.load(a, r, j0);
  double sum = 0.0;
#pragma unroll 1
  for (int i = first; i < a.pieces;) {
    const int64_t end = min(a.v, (i + 1) * a.piece);
    const bool last = j0 + kPiece >= end;
    const int at = last ? i + step : i;
    const int64_t then = last ? at * a.piece : j0 + kPiece;
    if (at < a.pieces) next.load(a, r, then);
    float p[8], q[8];
    now.values(a, r, j0, p, q);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += verify_left(p[k], q[k]);
    if (last) {
      take(i, wave_sum(sum));
      sum = 0.0;
    }
    i = at;
    j0 = then;
    now = next;
  }
}

// x of a whole of which 2^e is a share of 2^61 or more; one at least.
__device__ __forceinline__ uint64_t verify_count(double x, int e) {
  return x > 0.0 ? max((uint64_t)1, (uint64_t)__builtin_amdgcn_ldexp(x, e)) : 0;
}
__device__ __forceinline__ uint64_t verify_border(double x, int e) {
  const double y = __builtin_amdgcn_ldexp(x, e);
  return y > 0.0 ? (y < 0x1p63 ? (uint64_t)y : (uint64_t)1 << 63) : 0;
}

// The token that u falls on, by a whole wave; part[i]: the sum of piece i, up to 64 PER
// of them.  -1 where the row has no finite sum above zero.
template <bool HALF, int PER>
__device__ __forceinline__ int verify_draw(const VerifyArgs& a, VerifyRow& r, double u, const double* part) {
  const int lane = threadIdx.x & 63;
  const int per = (a.pieces + 63) / 64, i0 = lane * per;
  double x[PER];                         // this lane's pieces i0 ..
  auto add = [&] {
    double own = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) own += x[i];
    return wave_sum(own);
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = i < per && i0 + i < a.pieces ? part[i0 + i] : 0.0;
  double total = add();
  if (total == 0.0 && (r.two || r.without >= 0)) {
    // p nowhere above q: the token comes from p (rows that do not add up to one, or
    // a draft rejected by rounding alone; so seldom that one wave may do it)
    r.two = false;
    r.without = -1;
    verify_sums<HALF>(a, r, 0, 1, [&](int piece, double sum) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i < per && piece == i0 + i) x[i] = sum;
    });
    total = add();
  }
  const double border = u * total;
  if (!(total > 0.0 && total < __builtin_inf())) return -1;
  // the piece
  int e = 62 - __builtin_amdgcn_frexp_exp(total);
  uint64_t all, mine = 0;
  int last = -1;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint64_t c = verify_count(x[i], e);
    mine += c;
    if (c != 0) last = i;
  }
  constexpr uint64_t kLast = (uint64_t)1 << 63;   // u of 1 and more: the last token with a share
  uint64_t want = u < 1.0 ? verify_border(border, e) : kLast;
  uint64_t run = wave_before(mine, all);
  int at = last;
  uint64_t hit;
  if (want < all) {
    hit = __ballot(run <= want && want < run + mine);
    bool found = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      run += verify_count(x[i], e);
      if (!found && run > want) at = i, found = true;
    }
  } else {                               // by rounding, or kLast
    hit = (uint64_t)1 << (63 - __builtin_clzll(__ballot(last >= 0)));
  }
  const int winner = __builtin_ctzll(hit), place = __builtin_amdgcn_readlane(at, winner);
  double base = 0.0, own = 0.0;          // the sum before the piece; the piece's
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (lane < winner || (lane == winner && i < place)) base += x[i];
    if (i == place) own = x[i];
  }
  const double rest = border - wave_sum(base);
  // the token in it
  e = 62 - __builtin_amdgcn_frexp_exp(lane_of(own, winner));
  want = u < 1.0 ? verify_border(rest, e) : kLast;
  uint64_t before = 0;
  int token = -1;                        // this lane's last one with a share
  const int64_t piece = (int64_t)winner * per + place;
#pragma unroll 1
  for (int64_t j0 = piece * a.piece; j0 < min(a.v, (piece + 1) * a.piece); j0 += kPiece) {
    VerifyEight<HALF, true> eight;
    eight.load(a, r, j0);
    float p[8], q[8];
    eight.values(a, r, j0, p, q);
    uint64_t c[8];
    mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = verify_count(verify_left(p[i], q[i]), e);
      mine += c[i];
      if (c[i] != 0) token = (int)j0 + 8 * lane + i;
    }
    run = before + wave_before(mine, all);
    hit = __ballot(run <= want && want < run + mine);
    if (hit != 0) {
      bool found = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        run += c[i];
        if (!found && run > want) token = (int)j0 + 8 * lane + i, found = true;
      }
      return __builtin_amdgcn_readlane(token, __builtin_ctzll(hit));
    }
    before += all;
  }
  return (int)lane_of(wave_scan((uint32_t)(token + 1), 0u, [](uint32_t a, uint32_t b) { return max(a, b); }), 63) - 1;
}

__device__ __forceinline__ void verify_flag(const VerifyArgs& a, uint32_t flags) {
  if (flags != 0 && a.status) atomicOr(a.status, flags);
}

__device__ __forceinline__ void verify_store(const VerifyArgs& a, int b, const VerifyRow& r, int token) {
  a.next[b] = token;
  if (a.lens) a.lens[b] -= (int)(r.drafts - r.accepted);
  if (token < 0) verify_flag(a, QG_FLAG_NONFINITE);
}

// A workgroup a sequence.
template <bool HALF>
__global__ __launch_bounds__(1024) void verify_one_kernel(VerifyArgs a) {
  __shared__ double part[kVerifyOnePieces];
  const int wave = wave_id_uniform(), b = blockIdx.x;
  const float u = a.u_next[b];
  VerifyRow r;
  if (!verify_rows(a, b, r)) {           // the same in all waves
    if (threadIdx.x == 0) {              // nothing to verify, nothing to draw from
      a.accepted[b] = 0;
      a.next[b] = -1;
      verify_flag(a, QG_FLAG_INDEX);
    }
    return;
  }
  verify_find<HALF>(a, b, r);
  verify_sums<HALF>(a, r, wave, 16, [&](int piece, double sum) {
    if ((threadIdx.x & 63) == 0) part[piece] = sum;
  });
  __syncthreads();
  if (wave != 0) return;
  const int token = verify_draw<HALF, kVerifyOnePieces / 64>(a, r, (double)u, part);
  if (threadIdx.x != 0) return;
  a.accepted[b] = r.accepted;
  if (r.bad) verify_flag(a, QG_FLAG_INDEX);
  verify_store(a, b, r, token);
}

// Many workgroups a sequence, a piece or a few each wave; then a wave a sequence.
template <bool HALF>
__global__ __launch_bounds__(256) void verify_sums_kernel(VerifyArgs a) {
  const int b = blockIdx.y;
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  VerifyRow r;
  if (!verify_rows(a, b, r)) {
    if (first) a.accepted[b] = 0;
    return;
  }
  verify_find<HALF>(a, b, r);
  if (first) {
    a.accepted[b] = r.accepted;
    if (r.bad) verify_flag(a, QG_FLAG_INDEX);
  }
  verify_sums<HALF>(a, r, blockIdx.x * 4 + wave_id_uniform(), gridDim.x * 4, [&](int piece, double sum) {
    if ((threadIdx.x & 63) == 0) a.part[(size_t)b * a.pieces + piece] = sum;
  });
}

template <bool HALF, int PER>
__global__ __launch_bounds__(64) void verify_draw_kernel(VerifyArgs a) {
  const int b = blockIdx.x;
  const int accepted = __builtin_amdgcn_readfirstlane(a.accepted[b]);   // of the launch before, as the sums
  const float u = a.u_next[b];
  VerifyRow r;
  if (!verify_rows(a, b, r)) {
    if (threadIdx.x == 0) {
      a.next[b] = -1;
      verify_flag(a, QG_FLAG_INDEX);
    }
    return;
  }
  verify_at(a, b, accepted, r);
  const int token = verify_draw<HALF, PER>(a, r, (double)u, a.part + (size_t)b * a.pieces);
  if (threadIdx.x == 0) verify_store(a, b, r, token);
}

int64_t verify_piece(int64_t v) {
  int64_t c = kPiece;
  while ((v + c - 1) / c > kMaxPieces) c *= 2;
  return c;
}

// Whether one workgroup a sequence does it all.
bool verify_in_one(int64_t b, int64_t v) {
  // A short row, or sequences for every second CU: there one launch takes as long as the
  // two or less (kernels alone, fp32: one sequence of 32000 7.1 us against 3.6 + 3.0, 64 of
  // 40000 9.8 against 5.3 + 4.0; in bf16 61 of 32768 9.5 against 4.8 + 4.4; 128 of 131071
  // 27.3 against 20.4 + 4.7, 256 44.6 against 41.0 + 4.0; but 64 of 131071 27 against 13 + 4).
  if ((v + kPiece - 1) / kPiece > kVerifyOnePieces) return false;
  return v <= 40000 || b >= kCUs / 2;
}

int64_t verify_ws_bytes(int64_t b, int64_t v) {
  const int64_t c = verify_piece(v);
  return verify_in_one(b, v) ? 0 : b * ((v + c - 1) / c) * 8;
}

hipError_t launch_verify_drafts(VerifyArgs a, hipStream_t stream) {
  a.piece = verify_piece(a.v);
  a.pieces = (int)((a.v + a.piece - 1) / a.piece);
  auto on16 = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  a.whole = a.v % (a.half ? 8 : 4) == 0 && on16(a.target) && on16(a.draft);
  if (verify_in_one(a.b, a.v)) {
    if (a.half)
      hipLaunchKernelGGL((verify_one_kernel<true>), dim3(a.b), dim3(1024), 0, stream, a);
    else
      hipLaunchKernelGGL((verify_one_kernel<false>), dim3(a.b), dim3(1024), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t waves = (int64_t)a.b * a.pieces / (16 * kCUs);   // pieces a wave, 16 waves a CU
  const int per = (int)(waves < 1 ? 1 : waves > 4 ? 4 : waves);
  const dim3 grid((a.pieces + 4 * per - 1) / (4 * per), a.b);
  if (a.half)
    hipLaunchKernelGGL((verify_sums_kernel<true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((verify_sums_kernel<false>), grid, dim3(256), 0, stream, a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  if (a.half && a.pieces <= 256)
    hipLaunchKernelGGL((verify_draw_kernel<true, 4>), dim3(a.b), dim3(64), 0, stream, a);
  else if (a.half)
    hipLaunchKernelGGL((verify_draw_kernel<true, 16>), dim3(a.b), dim3(64), 0, stream, a);
  else if (a.pieces <= 256)
    hipLaunchKernelGGL((verify_draw_kernel<false, 4>), dim3(a.b), dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL((verify_draw_kernel<false, 16>), dim3(a.b), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
