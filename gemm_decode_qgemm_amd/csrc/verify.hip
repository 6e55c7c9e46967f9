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
// between tokens by a ten-thousandth of a likely token's share.
//
// Two launches over the one row that counts:
//   sums  every workgroup finds the sequence's first rejected draft (a few loads)
//         and adds up its 2048 or more tokens of that row; both the sum of
//         max(p - q, 0) and that of p, which stands in where the first is zero
//   draw  finds the part that holds the border, and the token in it
#include "layer_common.h"

namespace qg {

constexpr int kVerifyThreads = 256;

template <bool HALF>
__device__ __forceinline__ float prob(const void* p, size_t at) {
  if constexpr (HALF) return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
  return static_cast<const float*>(p)[at];
}

struct Row {                         // where the next token of a sequence comes from
  int64_t first, drafts;             // rows of the target: first .. first + drafts
  int accepted;
  int64_t p, q;                      // row of the target; of the draft, or -1
  int without;                       // the rejected token where drafts have no probabilities, or -1
  bool bad;                          // a drafted token outside the vocabulary
};

// Rows of sequence b, clipped to what there is.
__device__ __forceinline__ void verify_rows(const VerifyArgs& a, int b, int64_t& first, int64_t& drafts) {
  first = a.cu[b];
  int64_t end = a.cu[b + 1];
  first = first < 0 ? 0 : first;
  end = end > a.rows ? a.rows : end;
  drafts = end - first - 1;          // -1: a sequence without a row
  if (first - b < 0 || first - b + drafts > a.rows - a.b) drafts = -1;   // offsets that are not in order
}

// The row of the first rejected draft, or the one after the last; by whole waves.
template <bool HALF>
__device__ __forceinline__ void verify_at(const VerifyArgs& a, int b, int accepted, Row& r) {
  r.accepted = accepted;
  r.p = r.first + accepted;
  r.q = -1;
  r.without = -1;
  if (accepted < r.drafts) {
    const int64_t d = r.first - b + accepted;
    if (a.draft)
      r.q = d;
    else
      r.without = a.tokens[d];
  }
}

template <bool HALF>
__device__ __forceinline__ int verify_accepted(const VerifyArgs& a, int b, int64_t first, int64_t drafts, bool& bad) {
  const int lane = threadIdx.x & 63;
  bad = false;
  for (int64_t i0 = 0; i0 < drafts; i0 += 64) {
    const int64_t i = i0 + lane, d = first - b + i;
    bool ok = i >= drafts, out = false;
    if (i < drafts) {
      const int x = a.tokens[d];
      out = x < 0 || x >= a.v;
      if (!out) {
        const double p = (double)prob<HALF>(a.target, (size_t)(first + i) * a.v + x);
        const double q = a.draft ? (double)prob<HALF>(a.draft, (size_t)d * a.v + x) : 1.0;
        ok = (double)a.u[d] * q < p;
      }
    }
    const uint64_t no = __ballot(!ok);
    const int at = no ? __builtin_ctzll(no) : 64;
    bad = (__ballot(out) & (at < 64 ? ((uint64_t)2 << at) - 1 : ~(uint64_t)0)) != 0;
    if (no) return (int)(i0 + at);
  }
  return (int)(drafts < 0 ? 0 : drafts);
}

// What token j weighs: max(p - q, 0), where a NaN counts as 0; and max(p, 0).
template <bool HALF>
__device__ __forceinline__ void verify_weight(const VerifyArgs& a, const Row& r, int64_t j, double& left, double& whole) {
  const double p = (double)prob<HALF>(a.target, (size_t)r.p * a.v + j);
  const double q = r.q >= 0 ? (double)prob<HALF>(a.draft, (size_t)r.q * a.v + j) : 0.0;
  whole = fmax(p, 0.0);
  left = j == r.without ? 0.0 : fmax(p - q, 0.0);
}

__device__ __forceinline__ double wave_add(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

template <bool HALF>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a) {
  __shared__ double red[2][4];
  const int tid = threadIdx.x, b = blockIdx.y;
  Row r;
  verify_rows(a, b, r.first, r.drafts);
  if (r.drafts < 0) return;          // the same for the whole workgroup
  const int accepted = verify_accepted<HALF>(a, b, r.first, r.drafts, r.bad);
  verify_at<HALF>(a, b, accepted, r);
  double left = 0.0, whole = 0.0;
  const int64_t j1 = min(a.v, (int64_t)(blockIdx.x + 1) * a.chunk);
  for (int64_t j = (int64_t)blockIdx.x * a.chunk + tid; j < j1; j += kVerifyThreads) {
    double l, w;
    verify_weight<HALF>(a, r, j, l, w);
    left += l;
    whole += w;
  }
  left = wave_add(left);
  whole = wave_add(whole);
  if ((tid & 63) == 0) red[0][tid >> 6] = left, red[1][tid >> 6] = whole;
  __syncthreads();
  if (tid >= 2) return;
  a.part[((size_t)b * a.chunks + blockIdx.x) * 2 + tid] = (red[tid][0] + red[tid][1]) + (red[tid][2] + red[tid][3]);
  if (blockIdx.x == 0 && tid == 0) {
    a.accepted[b] = accepted;
    if (r.bad && a.status) atomicOr(a.status, QG_FLAG_INDEX);
  }
}

template <bool HALF>
__global__ __launch_bounds__(kVerifyThreads) void verify_draw_kernel(VerifyArgs a) {
  __shared__ double base_s;
  __shared__ int chunk_s, mode_s;
  __shared__ uint64_t wave_s[4];
  __shared__ int at_s[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id_uniform(), b = blockIdx.x;
  Row r;
  verify_rows(a, b, r.first, r.drafts);
  if (r.drafts < 0) {                // nothing to verify, nothing to draw from
    if (tid == 0) {
      a.accepted[b] = 0;
      a.next[b] = -1;
      if (a.status) atomicOr(a.status, QG_FLAG_INDEX);
    }
    return;
  }
  const int accepted = a.accepted[b];
  verify_at<HALF>(a, b, accepted, r);
  const double* const part = a.part + (size_t)b * a.chunks * 2;
  const double u = (double)a.u_next[b];
  if (tid == 0) {
    // One after another: the running sums never fall, so the part that the border is in has a sum above zero.
    int mode = 0;
    double total = 0.0;
    for (int s = 0; s < a.chunks; ++s) total += part[2 * s];
    if (total == 0.0) {
      mode = 1;
      for (int s = 0; s < a.chunks; ++s) total += part[2 * s + 1];
    }
    int chunk = -1;
    double base = 0.0, border = 0.0;
    if (total > 0.0 && total < __builtin_inf()) {
      border = u * total;
      double sum = 0.0;
      for (int s = 0; s < a.chunks; ++s) {
        const double x = part[2 * s + mode];
        if (x > 0.0) {               // the last one stays where u is 1 or more
          chunk = s;
          base = sum;
          if (sum + x > border) break;
        }
        sum += x;
      }
    }
    chunk_s = chunk;
    mode_s = mode;
    base_s = border - base;
  }
  __syncthreads();
  const int chunk = chunk_s;
  if (a.lens && tid == 0) a.lens[b] -= (int)(r.drafts - accepted);
  if (chunk < 0) {
    if (tid == 0) {
      a.next[b] = -1;
      if (a.status) atomicOr(a.status, QG_FLAG_NONFINITE);
    }
    return;
  }
  // Within the part, sums of whole numbers: exact, in any order.  A token counts
  // 2^61 times its share of the part, and at least one.
  const int mode = mode_s;
  const double all = part[2 * chunk + mode];
  const int e = 61 - ilogb(all);
  const double rest = ldexp(base_s, e);
  const uint64_t border = rest > 0.0 ? (rest < 0x1p63 ? (uint64_t)rest : (uint64_t)1 << 63) : 0;
  const int64_t j0 = (int64_t)chunk * a.chunk, j1 = min(a.v, j0 + a.chunk);
  const int per = (int)((a.chunk + kVerifyThreads - 1) / kVerifyThreads);
  auto count = [&](int64_t j) -> uint64_t {
    double l, w;
    verify_weight<HALF>(a, r, j, l, w);
    const double x = mode ? w : l;
    return x > 0.0 ? max((uint64_t)1, (uint64_t)ldexp(x, e)) : 0;
  };
  uint64_t mine = 0;
  int64_t last = -1;                 // this thread's last token with a share
  const int64_t t0 = j0 + (int64_t)tid * per, t1 = min(j1, t0 + per);
  for (int64_t j = t0; j < t1; ++j) {
    const uint64_t c = count(j);
    mine += c;
    if (c) last = j;
  }
  uint64_t sum = mine;               // running over the threads
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint64_t v = __shfl_up(sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 63) wave_s[wave] = sum;
  const uint64_t some = __ballot(last >= 0);
  if (lane == 0) at_s[wave] = some ? 64 * wave + 63 - __builtin_clzll(some) : -1;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += wave_s[w];
  const uint64_t before = sum - mine;
  const uint64_t end = wave_s[0] + wave_s[1] + wave_s[2] + wave_s[3];
  if (border >= end) {               // by rounding, or u of 1 and more: the last token with a share
    const int t = max(max(at_s[0], at_s[1]), max(at_s[2], at_s[3]));
    if (tid == t) a.next[b] = (int)last;
  } else if (before <= border && border < sum) {
    uint64_t run = before;
    for (int64_t j = t0; j < t1; ++j) {
      run += count(j);
      if (run > border) {
        a.next[b] = (int)j;
        break;
      }
    }
  }
}

// Tokens a workgroup adds up: 2048, more where a row would have over 128 parts.
int verify_chunk(int64_t v) {
  int64_t c = 2048;
  while ((v + c - 1) / c > 128) c *= 2;
  return (int)c;
}

hipError_t launch_verify_drafts(const VerifyArgs& a, hipStream_t stream) {
  if (a.half)
    hipLaunchKernelGGL((verify_sums_kernel<true>), dim3(a.chunks, a.b), dim3(kVerifyThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((verify_sums_kernel<false>), dim3(a.chunks, a.b), dim3(kVerifyThreads), 0, stream, a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  if (a.half)
    hipLaunchKernelGGL((verify_draw_kernel<true>), dim3(a.b), dim3(kVerifyThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((verify_draw_kernel<false>), dim3(a.b), dim3(kVerifyThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace qg
