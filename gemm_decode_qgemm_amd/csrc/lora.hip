// lora.hip -- the low-rank adapters of many requests beside a shared
// projection (qg_lora_add), up to 64 rows.
//
//   out[m] = y[m] + s_i (x[m] A_i^T) B_i^T,   i = ids[m]
// All products are exact bf16 by bf16 with fp32 sums: A and x are bf16, and the
// inner value s_i (x A_i^T) enters the second product as the sum of three bf16
// (24 bits), which costs matrix instructions only, of which there are plenty.
//
// Two launches, as the second product needs all of the first:
//   down  a workgroup owns 16 ranks of one adapter and a part of K; its waves take
//         64 k in turn and are summed in LDS; partial sums in fp32
//   up    a wave owns 64 columns of one adapter's B or more; its workgroup adds the
//         partial sums of the adapter's rows
// A unit is an adapter, or the rows' adapters where a batch has fewer rows than
// there are adapters: then the first row that names an adapter works for all of
// its rows, so that every adapter in use is read once.
//
// The matrix instruction (16x16x32) has the rows of an adapter on one side and up to
// 16 rows of x on the other.  A single row wastes 15/16 of it, which is
// nothing: the kernels are bound by reading A and B, and where these are small by
// latency.  Kernels alone, in bf16: one row, rank 16, 6656 to 256 columns 4.4 + 2.1 us; 41
// rows of 24 adapters to 8448 columns 5.4 + 4.4; 64 adapters of rank 64, 6656 to 39936
// columns 13.5 (54 MB, 4.0 TB/s) + 61.5 to 63.5 (337 MB, 5.3 to 5.5 TB/s; reads alone in
// this pattern take 53).  Many rows of one adapter go four at a time through the same
// workgroups: 64 rows, rank 16, 6656 to 8448 columns 27.6 us for both, to 39936 28.4.
#include <algorithm>

#include "layer_common.h"
#include "w4_common.h"

namespace qg {

constexpr int kLoraRows = QG_MAX_M;
constexpr int kLoraSplits = 4;         // parts of K, at most
constexpr int kLoraWaves = 8;          // of a workgroup of the first product
constexpr int kLoraStep = 256 * kLoraWaves;   // k of a workgroup whose loads are all in flight together

// The rows of unit `unit` as a mask, or 0 where it has none (or another unit
// works for them); `adapter` is theirs.
__device__ __forceinline__ uint64_t lora_rows(const LoraArgs& a, int unit, int& adapter) {
  const int lane = threadIdx.x & 63;
  const int id = lane < a.m ? a.ids[lane] : -1;
  const bool by_adapter = a.adapters < a.m;
  adapter = by_adapter ? unit : __builtin_amdgcn_readlane(id, unit);
  if (adapter < 0 || adapter >= a.adapters) return 0;
  const uint64_t mask = __ballot(id == adapter);
  return by_adapter || (mask != 0 && __builtin_ctzll(mask) == unit) ? mask : 0;
}

// The n-th set bit's row for lane n, by way of LDS: rows[0 .. count - 1].
__device__ __forceinline__ void lora_list(uint64_t mask, int* rows) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64 && (mask >> lane & 1) != 0) rows[__popcll(mask & (((uint64_t)1 << lane) - 1))] = lane;
}

template <int MT>
__device__ __forceinline__ void lora_down(const LoraArgs& a, int adapter, int count, const int* rows, int r0, int k0,
                                          int k1, float (*red)[16][17]) {
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4, wave = wave_id_uniform();
  const int rank = min(r0 + i, a.r - 1);
  const uint16_t* const w = a.a + ((size_t)adapter * a.r + rank) * a.k + 8 * q;
  const uint16_t* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = a.x + (size_t)rows[min(16 * t + i, count - 1)] * a.k + 8 * q;
  f32x4_t acc[MT] = {};
  constexpr int U = 8 / MT;
  for (int c = k0 + 64 * wave; c < k1; c += 32 * kLoraWaves * U) {   // whole 128-byte lines a wave
    u32x4_t wv[U], xv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wv[u] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int t = 0; t < MT; ++t) xv[u][t] = u32x4_t{0u, 0u, 0u, 0u};
      const int at = c + 64 * kLoraWaves * (u >> 1) + 32 * (u & 1);
      if (at + 8 * q < k1) {         // k is a multiple of 8
        wv[u] = *reinterpret_cast<const u32x4_t*>(w + at);
#pragma unroll
        for (int t = 0; t < MT; ++t) xv[u][t] = *reinterpret_cast<const u32x4_t*>(x[t] + at);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[u][t]),
                                                         __builtin_bit_cast(bf16x8_t, wv[u]), acc[t], 0, 0, 0);
  }
  // acc[t][e]: row 16 t + 4 q + e of the unit, rank r0 + i
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (t > 0) lds_barrier();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][4 * q + e][i] = acc[t][e];
    lds_barrier();
    const int m = threadIdx.x >> 4, r = threadIdx.x & 15;
    if (m < 16 && 16 * t + m < count && r0 + r < a.r) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kLoraWaves; w += 2) v += red[w][m][r] + red[w + 1][m][r];
      a.part[((size_t)blockIdx.z * a.m + rows[16 * t + m]) * a.r + r0 + r] = v;
    }
  }
}

__global__ __launch_bounds__(64 * kLoraWaves) void lora_down_kernel(LoraArgs a) {
  __shared__ float red[kLoraWaves][16][17];
  __shared__ int rows[kLoraRows];
  int adapter;
  const uint64_t mask = lora_rows(a, blockIdx.y, adapter);
  if (mask == 0) return;             // the same in all waves
  lora_list(mask, rows);
  lds_barrier();
  const int count = __popcll(mask);
  const int steps = (a.k + 127) >> 7;                    // of 128 k, shared out evenly
  const int k0 = 128 * (int)((int64_t)steps * blockIdx.z / a.splits);
  const int k1 = min(a.k, 128 * (int)((int64_t)steps * (blockIdx.z + 1) / a.splits));
  if (count <= 16)
    lora_down<1>(a, adapter, count, rows, 16 * blockIdx.x, k0, k1, red);
  else if (count <= 32)
    lora_down<2>(a, adapter, count, rows, 16 * blockIdx.x, k0, k1, red);
  else
    lora_down<4>(a, adapter, count, rows, 16 * blockIdx.x, k0, k1, red);
}

template <bool Y32>
__device__ __forceinline__ float lora_y(const LoraArgs& a, int row, int col) {
  const size_t at = (size_t)row * a.y_stride + col;
  return Y32 ? static_cast<const float*>(a.y)[at] : bf16_to_f32(static_cast<const uint16_t*>(a.y)[at]);
}

template <bool OUT32>
__device__ __forceinline__ void lora_store(const LoraArgs& a, int row, int col, float v) {
  const size_t at = (size_t)row * a.out_stride + col;
  if constexpr (OUT32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<uint16_t*>(a.out)[at] = (uint16_t)f32_to_bf16_rne(v);
}

// The workgroup's columns of a row without an adapter, by a wave: y as it is; NaN for
// an adapter that is not there.
template <bool Y32, bool OUT32>
__device__ __forceinline__ void lora_rest(const LoraArgs& a, int m) {
  const int lane = threadIdx.x & 63;
  if (m >= a.m) return;
  const int id = a.ids[m];
  const bool bad = id >= a.adapters;
  if (id >= 0 && !bad) return;
  if (bad && a.status && blockIdx.x == 0 && lane == 0) atomicOr(a.status, QG_FLAG_INDEX);
  if (!bad && a.y == a.out) return;    // in place there is nothing to do
  for (int c0 = blockIdx.x * 256; c0 < a.n; c0 += gridDim.x * 256) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = bad ? __uint_as_float(0x7fc00000u) : lora_y<Y32>(a, m, min(c0 + 64 * j + lane, a.n - 1));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + 64 * j + lane < a.n) lora_store<OUT32>(a, m, c0 + 64 * j + lane, v[j]);
  }
}

// 64 columns of B, 4 tiles of 16, as a wave's operands; zeros past its view.  An operand
// holds PACK tiles side by side where that many ranks are all there are: 16 or 8.
template <int RS, int PACK>
struct LoraB {
  static constexpr int kOps = 4 / PACK;
  u32x4_t w[kOps][RS];

  static __device__ __forceinline__ int tile(int t) { return PACK * t + (threadIdx.x >> 4 & 3) / kOps; }   // of a lane
  static __device__ __forceinline__ int rank(int s) { return 32 * s + 8 * ((threadIdx.x >> 4 & 3) % kOps); }
  __device__ __forceinline__ void load(const BufView& b, int r, int col) {
    const uint32_t row = 2u * (uint32_t)r, at = (uint32_t)(col + 16 * tile(0) + (threadIdx.x & 15)) * row;
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const uint32_t from = rank(s) < r ? at + 2u * rank(s) : 0xfffffff0u - 64u * row;
#pragma unroll
      for (int t = 0; t < kOps; ++t) w[t][s] = b.b128<false>(from + 16u * PACK * t * row);
    }
  }
};

// 4 rows of y or out as views of their n columns.
struct LoraRows {
  __amdgpu_buffer_rsrc_t row[4];
  __device__ __forceinline__ LoraRows(const void* base, bool f32, int64_t stride, const int (&rows)[4], int part, int n) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t at = (int64_t)rows[m] * stride;
      row[m] = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(static_cast<const char*>(base) + at * (f32 ? 4 : 2)), (short)0,
          m < part ? n * (f32 ? 4 : 2) : 0, 0x00020000);
    }
  }
  template <bool F32>
  __device__ __forceinline__ float load(int m, int col) const {
    if constexpr (F32) return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row[m], 4 * col, 0, 0));
    return bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row[m], 2 * col, 0, 0));
  }
  template <bool F32>
  __device__ __forceinline__ void store(int m, int col, float v) const {
    if constexpr (F32)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), row[m], 4 * col, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16_rne(v), row[m], 2 * col, 0, 0);
  }
};

// Four rows' first product, scaled, as sums of three bf16: LDS of a workgroup.
template <int RS>
struct LoraInner {
  static constexpr int kRanks = 32 * RS, kRow = kRanks + 8;        // rows off the same banks
  static constexpr int kEach = (4 * kRanks + 255) / 256;            // values a thread
  uint16_t v[3][4][kRow];

  struct Parts { float f[kEach][kLoraSplits]; };
  static __device__ __forceinline__ void place(int j, int& m, int& rank) {
    const int at = (int)threadIdx.x + 256 * j;
    m = at / kRanks, rank = at % kRanks;
  }
  static __device__ __forceinline__ Parts load(const LoraArgs& a, const BufView& pv, const int (&rows)[4]) {
    Parts p;
    // (as registers: an array that is picked from would go to LDS)
    const int r0 = __builtin_amdgcn_readfirstlane(rows[0]), r1 = __builtin_amdgcn_readfirstlane(rows[1]);
    const int r2 = __builtin_amdgcn_readfirstlane(rows[2]), r3 = __builtin_amdgcn_readfirstlane(rows[3]);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      int m, rank;
      place(j, m, rank);
      const int row = (m & 2) ? ((m & 1) ? r3 : r2) : ((m & 1) ? r1 : r0);
      uint32_t at = rank < a.r ? 4u * (uint32_t)(row * a.r + rank) : 0xf0000000u;   // past the view: zeros
#pragma unroll
      for (int s = 0; s < kLoraSplits; ++s, at += 4u * (uint32_t)(a.m * a.r))
        p.f[j][s] = s < a.splits ? __uint_as_float(pv.b32(at)) : 0.0f;   // uniform
    }
    return p;
  }
  __device__ __forceinline__ void store(const Parts& p, int r, float scale) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      int m, rank;
      place(j, m, rank);
      if (m >= 4) continue;
      float f = p.f[j][0];
#pragma unroll
      for (int s = 1; s < kLoraSplits; ++s) f += p.f[j][s];
      f = rank < r ? f * scale : 0.0f;         // (an infinite scale times no rank is no NaN)
      // The first part is rounded towards zero where to nearest could give bf16's infinity: the
      // 16 bits behind it fill the other two as the rest of a rounded one does.
      const bool huge = fabsf(f) > 0x1p127f, inf = fabsf(f) == __builtin_inff();
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const uint32_t h = u == 0 && huge ? __float_as_uint(f) >> 16 : f32_to_bf16_rne(f) & 0xffffu;
        v[u][m][rank] = (uint16_t)h;
        f = inf ? 0.0f : f - __uint_as_float(h << 16);   // (infinite: all in the first)
      }
    }
  }
};

// RS steps of 32 ranks.  A wave takes TILES times 64 columns, and 4 rows at a time: the
// operand repeats them, so that lane (i, q) has all four for column i of every tile and
// takes tile q, 64 neighbouring columns a row.  (16 rows at a time would take a quarter of
// the matrix instructions, of which there are plenty, and touch 16 columns of a row
// at a time.)  The waves of a workgroup share what they need of the first product, each
// its part of the sums, by way of LDS; their loads of B are on the way meanwhile.
template <int RS, int PACK, int TILES, bool Y32, bool OUT32>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  __shared__ __attribute__((aligned(16))) LoraInner<RS> inner_s[2];   // in turn: a barrier each
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4, wave = wave_id_uniform();
  const int units = min(a.m, a.adapters);
  if ((int)blockIdx.y >= units) {
    lora_rest<Y32, OUT32>(a, 4 * ((int)blockIdx.y - units) + wave);
    return;
  }
  const int col = TILES * (blockIdx.x * 256 + 64 * wave);
  int adapter;
  uint64_t mask = lora_rows(a, blockIdx.y, adapter);
  if (mask == 0) return;               // the same in all waves; one past the columns goes on, for the barriers
  const BufView bv(a.b + (size_t)adapter * a.n * a.r, a.n * a.r * 2);
  const BufView pv(a.part, a.splits * a.m * a.r * 4);
  const float scale = a.scales ? a.scales[adapter] : 1.0f;
  int rows[4], some;
  auto next_rows = [&] {
    some = 0;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      rows[m] = m > 0 ? rows[m - 1] : 0;
      if (mask == 0) continue;
      rows[m] = __builtin_ctzll(mask);
      mask &= mask - 1;
      ++some;
    }
  };
  next_rows();
  typename LoraInner<RS>::Parts parts = LoraInner<RS>::load(a, pv, rows);   // first: waited for first
  using Ops = LoraB<RS, PACK>;
  Ops b[TILES];
#pragma unroll
  for (int c = 0; c < TILES; ++c) b[c].load(bv, a.r, col + 64 * c);
  for (int turn = 0;; turn ^= 1) {
    const LoraRows ys(a.y, Y32, a.y_stride, rows, some, a.n), os(a.out, OUT32, a.out_stride, rows, some, a.n);
    float y[TILES][4];
#pragma unroll
    for (int c = 0; c < TILES; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) y[c][m] = ys.load<Y32>(m, col + 64 * c + lane);
    LoraInner<RS>& inner = inner_s[turn];
    inner.store(parts, a.r, scale);
    lds_barrier();
#pragma unroll
    for (int c = 0; c < TILES; ++c) {
      f32x4_t acc[Ops::kOps] = {};
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int u = 2; u >= 0; --u) {
          const u32x4_t low = *reinterpret_cast<const u32x4_t*>(&inner.v[u][i & 3][Ops::rank(s)]);
#pragma unroll
          for (int t = 0; t < Ops::kOps; ++t) {
            // rows 4 T .. 4 T + 3 of the product are tile T's, which for the other tiles' ranks are zero
            const u32x4_t x = PACK == 1 || i >> 2 == Ops::tile(t) ? low : u32x4_t{0u, 0u, 0u, 0u};
            f32x4_t& to = acc[PACK == 1 ? t : 0];
            to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x),
                                                         __builtin_bit_cast(bf16x8_t, b[c].w[t][s]), to, 0, 0, 0);
          }
        }
      f32x4_t v = acc[0];              // of tile q
      if constexpr (PACK == 1)
#pragma unroll
        for (int m = 0; m < 4; ++m) v[m] = q < 2 ? (q == 0 ? v[m] : acc[1][m]) : (q == 2 ? acc[2][m] : acc[3][m]);
      bool none = false;
#pragma unroll
      for (int m = 0; m < 4; ++m) none |= v[m] != v[m];
      // A NaN may come of a weight that is infinite, times an inner value's second or third
      // part, or times the zeros between neighbouring tiles: every tile by itself, and a
      // sum that is still none from the first parts alone.
      if (__ballot(none) != 0) {
#pragma unroll 1
        for (int p = 0; p < PACK; ++p) {
          const bool own = q / Ops::kOps == p;
          const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int t = 0; t < Ops::kOps; ++t) {
            f32x4_t one = {}, some_of_it = {};
#pragma unroll
            for (int s = 0; s < RS; ++s)
#pragma unroll
              for (int u = 2; u >= 0; --u) {
                const u32x4_t low = *reinterpret_cast<const u32x4_t*>(&inner.v[u][i & 3][Ops::rank(s)]);
                const bf16x8_t x = __builtin_bit_cast(bf16x8_t, PACK == 1 || own ? low : zero);
                const bf16x8_t w = __builtin_bit_cast(bf16x8_t, PACK == 1 || own ? b[c].w[t][s] : zero);
                one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, one, 0, 0, 0);
                if (u == 0) some_of_it = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, some_of_it, 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);   // seldom here: no registers for it
              }
            if (q == PACK * t + p)
#pragma unroll
              for (int m = 0; m < 4; ++m) v[m] = one[m] != one[m] ? some_of_it[m] : one[m];
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) os.store<OUT32>(m, col + 64 * c + lane, y[c][m] + v[m]);
    }
    if (mask == 0) return;
    next_rows();
    parts = LoraInner<RS>::load(a, pv, rows);
  }
}

int lora_splits(int64_t m, int64_t k, int64_t r, int64_t adapters) {
  // Parts of K: a step each while that gives two workgroups a CU.
  const int64_t units = std::min(m, adapters) * ((r + 15) / 16), steps = (k + kLoraStep - 1) / kLoraStep;
  return (int)std::max<int64_t>(1, std::min<int64_t>({steps, kLoraSplits, (2 * kCUs + units - 1) / units}));
}

hipError_t launch_lora_add(LoraArgs a, hipStream_t stream) {
  const int units = std::min(a.m, a.adapters);
  hipLaunchKernelGGL(lora_down_kernel, dim3((a.r + 15) / 16, units, a.splits), dim3(64 * kLoraWaves), 0, stream, a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  const int types = (a.y_f32 ? 2 : 0) + (a.out_f32 ? 1 : 0);
#define QG_LORA(RS, PACK, TILES)                                                                          \
  {                                                                                                       \
    const dim3 grid((a.n + 256 * TILES - 1) / (256 * TILES), units + (a.m + 3) / 4), block(256);          \
    switch (types) {                                                                                      \
      case 0: hipLaunchKernelGGL((lora_up_kernel<RS, PACK, TILES, false, false>), grid, block, 0, stream, a); break; \
      case 1: hipLaunchKernelGGL((lora_up_kernel<RS, PACK, TILES, false, true>), grid, block, 0, stream, a); break;  \
      case 2: hipLaunchKernelGGL((lora_up_kernel<RS, PACK, TILES, true, false>), grid, block, 0, stream, a); break;  \
      case 3: hipLaunchKernelGGL((lora_up_kernel<RS, PACK, TILES, true, true>), grid, block, 0, stream, a); break;   \
    }                                                                                                     \
  }
  // Ranks of 8 and 16, which most adapters have, fill an operand with neighbouring tiles
  // (without: 64 adapters of 131072 columns, rank 8 66 us, rank 16 75).  Where 64
  // columns a wave make up four rounds of 16 waves a CU, a wave takes 256 or 128 (rank 8: 32 us
  // against 56, 16384 columns 10.3 against 11.9; rank 16: 53 against 62, 11.7 to 12.9 against
  // 12.4; 8192 columns 11 all).  Larger operands take the registers that hide latency: at
  // rank 64 128 columns a wave 65 us against 61 at 39936, at rank 128 125 against 116.
  const bool many = (int64_t)units * ((a.n + 63) / 64) >= 4 * 16 * kCUs;
  if (a.r == 8 && many)
    QG_LORA(1, 4, 4)
  else if (a.r == 8)
    QG_LORA(1, 4, 1)
  else if (a.r == 16 && many)
    QG_LORA(1, 2, 2)
  else if (a.r == 16)
    QG_LORA(1, 2, 1)
  else if (a.r <= 32)
    QG_LORA(1, 1, 1)
  else if (a.r <= 64)
    QG_LORA(2, 1, 1)
  else if (a.r <= 128)
    QG_LORA(4, 1, 1)
  else
    QG_LORA(8, 1, 1)
#undef QG_LORA
  return hipGetLastError();
}

}  // namespace qg
