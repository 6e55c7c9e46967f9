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

namespace qg {

constexpr int kLoraRows = QG_MAX_M;

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
  constexpr int U = MT == 1 ? 4 : 2;
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
    if (t > 0) __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][4 * q + e][i] = acc[t][e];
    __syncthreads();
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
  __syncthreads();
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

__device__ __forceinline__ float lora_y(const LoraArgs& a, int row, int col) {
  const size_t at = (size_t)row * a.y_stride + col;
  return a.y_f32 ? static_cast<const float*>(a.y)[at] : bf16_to_f32(static_cast<const uint16_t*>(a.y)[at]);
}

__device__ __forceinline__ void lora_store(const LoraArgs& a, int row, int col, float v) {
  const size_t at = (size_t)row * a.out_stride + col;
  if (a.out_f32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<uint16_t*>(a.out)[at] = (uint16_t)f32_to_bf16_rne(v);
}

// RS steps of 32 ranks, NB tiles of 16 columns a wave.
template <int RS>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  constexpr int NB = RS >= 4 ? 8 / RS : 4;
  constexpr int COLS = 64 * NB;                  // of a workgroup
  constexpr int ROWS = RS > 4 ? 32 : 64;         // at a time, for LDS
  constexpr int LD = 32 * RS + 8;                // bf16 apart: operand reads on distinct banks
  __shared__ __attribute__((aligned(16))) uint16_t low[3][ROWS][LD];
  __shared__ int rows[kLoraRows];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4, wave = wave_id_uniform();
  const int units = gridDim.y - 1;
  const int n0 = blockIdx.x * COLS;
  if ((int)blockIdx.y == units) {                // rows without an adapter
    for (int m = 0; m < a.m; ++m) {
      const int id = a.ids[m];
      if (id >= 0 && id < a.adapters) continue;
      const bool bad = id >= a.adapters;
      if (bad && a.status && blockIdx.x == 0 && tid == 0) atomicOr(a.status, QG_FLAG_INDEX);
      for (int c = n0 + tid; c < min(n0 + COLS, a.n); c += 256)
        lora_store(a, m, c, bad ? __uint_as_float(0x7fc00000u) : lora_y(a, m, c));
    }
    return;
  }
  int adapter;
  const uint64_t mask = lora_rows(a, blockIdx.y, adapter);
  if (mask == 0) return;                         // the same in all waves
  const int count = __popcll(mask);
  lora_list(mask, rows);
  u32x4_t w[NB][RS];                             // B, on its way while the partial sums are added
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const int col = min(n0 + 16 * (NB * wave + b) + i, a.n - 1), rank = 32 * s + 8 * q;
      w[b][s] = u32x4_t{0u, 0u, 0u, 0u};
      if (rank < a.r) w[b][s] = *reinterpret_cast<const u32x4_t*>(a.b + ((size_t)adapter * a.n + col) * a.r + rank);
    }
  __syncthreads();
  const float scale = a.scales ? a.scales[adapter] : 1.0f;
  for (int m0 = 0; m0 < count; m0 += ROWS) {
    if (m0 > 0) __syncthreads();
    const int part = min(ROWS, count - m0);
    for (int at = tid; at < part * 32 * RS; at += 256) {
      const int m = at / (32 * RS), r = at % (32 * RS);
      float v = 0.0f;
      if (r < a.r)
        for (int s = 0; s < a.splits; ++s) v += a.part[((size_t)s * a.m + rows[m0 + m]) * a.r + r];
      v = r < a.r ? v * scale : 0.0f;
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const uint32_t h = f32_to_bf16_rne(v);
        low[u][m][r] = (uint16_t)h;
        v = (h & 0x7fffu) < 0x7f80u ? v - bf16_to_f32(h) : 0.0f;   // an infinity is whole in the first
      }
    }
    __syncthreads();
    for (int t = 0; t < part; t += 16) {
      f32x4_t acc[NB] = {};
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int u = 2; u >= 0; --u) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(&low[u][min(t + i, part - 1)][32 * s + 8 * q]);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                             __builtin_bit_cast(bf16x8_t, w[b][s]), acc[b], 0, 0, 0);
        }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = t + 4 * q + e, col = n0 + 16 * (NB * wave + b) + i;
          if (m < part && col < a.n) lora_store(a, rows[m0 + m], col, lora_y(a, rows[m0 + m], col) + acc[b][e]);
        }
    }
  }
}

int lora_splits(int64_t m, int64_t k, int64_t r, int64_t adapters) {
  // Two workgroups a CU, of at least four steps of 128 k each.
  const int64_t units = std::min(m, adapters) * ((r + 15) / 16), steps = (k + 127) / 128;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(2 * kCUs + units - 1) / units, (steps + 3) / 4, 16}));
}

hipError_t launch_lora_add(const LoraArgs& a, hipStream_t stream) {
  const int units = std::min(a.m, a.adapters);
  hipLaunchKernelGGL(lora_down_kernel, dim3((a.r + 15) / 16, units, a.splits), dim3(256), 0, stream, a);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
#define QG_LORA(RS)                                                                                           \
  hipLaunchKernelGGL((lora_up_kernel<RS>), dim3((a.n + 64 * (RS >= 4 ? 8 / RS : 4) - 1) / (64 * (RS >= 4 ? 8 / RS : 4)), \
                                                units + 1), dim3(256), 0, stream, a)
  if (a.r <= 32)
    QG_LORA(1);
  else if (a.r <= 64)
    QG_LORA(2);
  else if (a.r <= 128)
    QG_LORA(4);
  else
    QG_LORA(8);
#undef QG_LORA
  return hipGetLastError();
}

}  // namespace qg
