// lora.hip -- the low-rank adapters of many requests beside a shared
// projection (qg_lora_add), up to 64 rows.
//
//   out[m] = y[m] + s_i (x[m] A_i^T) B_i^T,   i = ids[m]
// All products are exact bf16 by bf16 with fp32 sums: A and x are bf16, and the
// inner value s_i (x A_i^T) enters the second product as the sum of three bf16
// (24 bits), which costs matrix instructions only, of which there are plenty.
//
// Two launches, as the second product needs all of the first:
//   down  a workgroup owns 16 ranks of one adapter and a part of K; its four
//         waves take 32 k in turn and are summed in LDS; partial sums in fp32
//   up    a workgroup owns columns of one adapter's B; it adds the partial sums
//         of the adapter's rows, then its waves take 16 columns at a time
// A unit is an adapter, or the rows' adapters where a batch has fewer rows than
// there are adapters: then the first row that names an adapter works for all of
// its rows, so that every adapter in use is read once.
//
// The matrix instruction (16x16x32) has the rows of an adapter on one side and up to
// 16 rows of x on the other.  A single row wastes 15/16 of it, which is
// nothing: the kernels are bound by reading A and B.
#include <algorithm>

#include "layer_common.h"
#include "w4_common.h"

namespace qg {

constexpr int kLoraRows = QG_MAX_M;
constexpr int kLoraSplits = 16;        // of K, at most
constexpr int kLoraStep = 1024;        // k of a workgroup whose loads are all in flight together

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
  constexpr int U = MT == 1 ? kLoraStep / 128 : MT == 2 ? 4 : 2;
  for (int c = k0 + 32 * wave; c < k1; c += 128 * U) {
    u32x4_t wv[U], xv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wv[u] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int t = 0; t < MT; ++t) xv[u][t] = u32x4_t{0u, 0u, 0u, 0u};
      const int at = c + 128 * u;
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
    if (16 * t + m < count && r0 + r < a.r)
      a.part[((size_t)blockIdx.z * a.m + rows[16 * t + m]) * a.r + r0 + r] =
          (red[0][m][r] + red[1][m][r]) + (red[2][m][r] + red[3][m][r]);
  }
}

__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a) {
  __shared__ float red[4][16][17];
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

// 64 columns of B, 4 tiles of 16, as a wave's operands; zeros past its view.
template <int RS>
struct LoraB {
  u32x4_t w[4][RS];

  __device__ __forceinline__ void load(const BufView& b, int r, int col) {
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    const uint32_t row = 2u * (uint32_t)r, at = (uint32_t)(col + i) * row + 16u * q;
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const uint32_t from = 32 * s + 8 * q < r ? at + 64u * s : 0xfffffff0u - 64u * row;
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t][s] = b.b128<false>(from + 16u * t * row);
    }
  }
};

// 4 rows of y or out as views of their n columns.
struct LoraRows {
  __amdgpu_buffer_rsrc_t row[4];
  __device__ __forceinline__ LoraRows(const void* base, bool f32, int64_t stride, const int* rows, int part, int n) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t at = (int64_t)__builtin_amdgcn_readfirstlane(rows[min(m, part - 1)]) * stride;
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

// RS steps of 32 ranks.  A wave takes 64 columns at a time, B of the next ones in
// flight, and 4 rows at a time: the operand repeats them, so that lane (i, q) has all
// four for column i of every tile and takes tile q, 64 neighbouring columns a row.
// (16 rows at a time would take a quarter of the matrix instructions, of which there
// are plenty, and touch 16 columns of a row at a time.)
#ifndef QG_LS
#define QG_LS 4
#define QG_LD 8
#endif
#ifdef QG_LW
#define QG_WP __attribute__((amdgpu_waves_per_eu(QG_LW)))
#else
#define QG_WP
#endif
template <int RS, bool Y32, bool OUT32>
__global__ __launch_bounds__(256) QG_WP void lora_up_kernel(LoraArgs a) {
  constexpr int LD = 32 * RS + 8;                // bf16 apart: operand reads on distinct banks
  __shared__ __attribute__((aligned(16))) uint16_t low[3][16][LD];
  __shared__ int rows[kLoraRows];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4, wave = wave_id_uniform();
  const int units = min(a.m, a.adapters);
  const int first = blockIdx.x * 256 + 64 * wave, stride = gridDim.x * 256;   // this wave's columns
  if ((int)blockIdx.y >= units) {
    lora_rest<Y32, OUT32>(a, 4 * ((int)blockIdx.y - units) + wave);
    return;
  }
  int adapter;
  const uint64_t mask = lora_rows(a, blockIdx.y, adapter);
  if (mask == 0) return;                         // the same in all waves
  const int count = __popcll(mask);
  lora_list(mask, rows);
  const BufView b(a.b + (size_t)adapter * a.n * a.r, a.n * a.r * 2);
  LoraB<RS> w0;
  w0.load(b, a.r, first);                    // on its way while the first product's parts are added
  lds_barrier();
  const float scale = a.scales ? a.scales[adapter] : 1.0f;
  for (int m0 = 0; m0 < count; m0 += 16) {
    const int part = min(16, count - m0);
    const int* const mine = rows + m0;
    if (m0 > 0) {
      lds_barrier();
      w0.load(b, a.r, first);
    }
    const LoraRows y0(a.y, Y32, a.y_stride, mine, min(part, 4), a.n);
    float y[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = y0.load<Y32>(m, first + lane);
#pragma unroll 1
    for (int at = tid; at < part * 32 * RS; at += 256) {
      const int m = at / (32 * RS), r = at % (32 * RS);
      float v = 0.0f;
      if (r < a.r) {
        float t[kLoraSplits];                    // all on their way together
        const float* const p = a.part + (size_t)mine[m] * a.r + r;
#pragma unroll
        for (int s = 0; s < kLoraSplits; ++s) t[s] = s < a.splits ? p[(size_t)s * a.m * a.r] : 0.0f;
#pragma unroll
        for (int s = 0; s < kLoraSplits; ++s) v += t[s];
        v *= scale;
      }
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const uint32_t h = f32_to_bf16_rne(v);
        low[u][m][r] = (uint16_t)h;
        v = (h & 0x7fffu) < 0x7f80u ? v - bf16_to_f32(h) : 0.0f;   // an infinity is whole in the first
      }
    }
    lds_barrier();
    auto step = [&](const LoraB<RS>& w, int col) {
      for (int g = 0; g < part; g += 4) {
        const int some = min(part - g, 4);
        const LoraRows ys(a.y, Y32, a.y_stride, mine + g, some, a.n);
        if (g > 0) {
#pragma unroll
          for (int m = 0; m < 4; ++m) y[m] = ys.load<Y32>(m, col + lane);
        }
        f32x4_t acc[4] = {};
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
          for (int u = 2; u >= 0; --u) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(&low[u][g + min(i & 3, some - 1)][32 * s + 8 * q]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                               __builtin_bit_cast(bf16x8_t, w.w[t][s]), acc[t], 0, 0, 0);
          }
        const LoraRows os(a.out, OUT32, a.out_stride, mine + g, some, a.n);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float v = q < 2 ? (q == 0 ? acc[0][m] : acc[1][m]) : (q == 2 ? acc[2][m] : acc[3][m]);
          os.store<OUT32>(m, col + lane, y[m] + v);
        }
      }
    };
    for (int col = first; col < a.n; col += stride) {
      const int next = col + stride;
      if constexpr (RS <= 4) {
        LoraB<RS> w1;
        if (next < a.n) w1.load(b, a.r, next);
        step(w0, col);
        w0 = w1;
      } else {                                   // B takes the registers of two: no next one in flight
        step(w0, col);
        if (next < a.n) w0.load(b, a.r, next);
      }
      if (next < a.n)
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] = y0.load<Y32>(m, next + lane);
    }
  }
}

int lora_splits(int64_t m, int64_t k, int64_t r, int64_t adapters) {
  (void)m, (void)r, (void)adapters;
  return (int)std::min<int64_t>(kLoraSplits, (k + kLoraStep - 1) / kLoraStep);
}

hipError_t launch_lora_add(LoraArgs a, hipStream_t stream) {
  const int units = std::min(a.m, a.adapters);
  hipLaunchKernelGGL(lora_down_kernel, dim3((a.r + 15) / 16, units, a.splits), dim3(256), 0, stream, a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  // Steps a wave: up to 4 while eight workgroups a CU are left.
  const int blocks = (a.n + 255) / 256;
  a.steps = std::max(1, std::min(QG_LS, (int)((int64_t)units * blocks / (QG_LD * kCUs))));
  const dim3 grid((blocks + a.steps - 1) / a.steps, units + (a.m + 3) / 4);
  const int types = (a.y_f32 ? 2 : 0) + (a.out_f32 ? 1 : 0);
#define QG_LORA(RS)                                                                                    \
  switch (types) {                                                                                     \
    case 0: hipLaunchKernelGGL((lora_up_kernel<RS, false, false>), grid, dim3(256), 0, stream, a); break; \
    case 1: hipLaunchKernelGGL((lora_up_kernel<RS, false, true>), grid, dim3(256), 0, stream, a); break;  \
    case 2: hipLaunchKernelGGL((lora_up_kernel<RS, true, false>), grid, dim3(256), 0, stream, a); break;  \
    case 3: hipLaunchKernelGGL((lora_up_kernel<RS, true, true>), grid, dim3(256), 0, stream, a); break;   \
  }
  if (a.r <= 32)
    QG_LORA(1)
  else if (a.r <= 64)
    QG_LORA(2)
  else if (a.r <= 128)
    QG_LORA(4)
  else
    QG_LORA(8)
#undef QG_LORA
  return hipGetLastError();
}

}  // namespace qg
