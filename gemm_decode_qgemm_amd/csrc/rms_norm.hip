// rms_norm.hip -- a sub-layer's output added to the residual stream and the
// RMS norm of the sum, in one pass over both (qg_rms_norm, qg_rms_norm_q8).
//
//   r = x + residual;   y = r * rsqrt(mean(r^2) + eps) * w
// in fp32: the norm takes the sum as it is before r is rounded to the stream's
// type, and y is rounded once, to bf16 or to 8-bit codes with the scales of the
// W4A8 linears (act_q8.h).
//
// Mapping: a row is kept in the registers of the threads that read it, 8
// channels a thread and chunk, so that it is read once and the sums are the only
// thing that waits: a wave per row up to 2048 channels, else a workgroup.  The
// 32 channels of a scale group are the chunks of four neighbouring lanes.  Long prompts
// are bound by memory (16383 rows of 4096 on a 32-bit stream, 8-bit rows: 402 MB read
// and 344 written in 130 to 134 us, 5.6 to 5.7 TB/s), few rows by latency (one row of
// 6656 3.2 us, 61 in 8 bits 5.2), rows much narrower than a wave's 512 channels by the
// lanes that have none (65536 rows of 64 16 us where a copy takes 3.5, of 256 18 for 14).
#include "act_q8.h"
#include "layer_common.h"

namespace qg {

template <bool F32>
struct Raw {                         // 8 channels as they lie in memory
  u32x4_t a[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    if constexpr (F32) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(base) + at);
      a[0] = p[0];
      a[1] = p[1];
    } else {
      a[0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + at);
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (F32) return __uint_as_float(a[e >> 2][e & 3]);
    return __uint_as_float((e & 1) ? a[0][e >> 1] & 0xffff0000u : a[0][e >> 1] << 16);
  }
};

// Sum or NaN-keeping maximum over the T threads of a row; `red` is not used again
// before the next barrier.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const float u = __shfl_xor(v, o);
    v = MAX ? nmax(v, u) : v + u;
  }
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = MAX ? nmax(v, red[w]) : v + red[w];
  }
  return v;
}

// X32: x in fp32; RES: 0 no residual, 1 bf16, 2 fp32; CH chunks of 8 channels a thread.
template <int T, int CH, bool X32, int RES>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rms_norm_kernel(RmsNormArgs a) {
  __shared__ float red[3][16];
  const int tid = T == 64 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int64_t row = T == 64 ? (int64_t)blockIdx.x * 4 + wave_id_uniform() : (int64_t)blockIdx.x;
  if (row >= a.rows) return;         // T == 64: waves of a workgroup share nothing
  const int chunks = a.h >> 3;
  Raw<X32> xr[CH];
  Raw<RES == 2> rr[CH];
  Raw<false> wr[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = tid + T * j;
    if (c >= chunks) continue;
    xr[j].load(a.x, (size_t)row * a.x_stride + 8 * c);
    if constexpr (RES != 0) rr[j].load(a.res, (size_t)row * a.res_stride + 8 * c);
  }
  if (a.w) {
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (tid + T * j < chunks) wr[j].load(a.w, 8 * (tid + T * j));
  }
  float v[CH][8];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = tid + T * j;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[j][e] = 0.0f;
      if (c < chunks) {
        v[j][e] = xr[j].get(e);
        if constexpr (RES != 0) v[j][e] += rr[j].get(e);
      }
      ss = __builtin_fmaf(v[j][e], v[j][e], ss);
    }
    if constexpr (RES != 0) {
      if (c >= chunks) continue;
      const size_t at = (size_t)row * a.h + 8 * c;
      if constexpr (RES == 2) {
        f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.res_out) + at);
        p[0] = f32x4_t{v[j][0], v[j][1], v[j][2], v[j][3]};
        p[1] = f32x4_t{v[j][4], v[j][5], v[j][6], v[j][7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.res_out) + at) =
            u32x4_t{pack_bf16(v[j][0], v[j][1]), pack_bf16(v[j][2], v[j][3]), pack_bf16(v[j][4], v[j][5]),
                    pack_bf16(v[j][6], v[j][7])};
      }
    }
  }
  ss = row_reduce<T, false>(ss, red[0]);
  const float n = (float)a.h;
  const float mean = ss / n + a.eps;
  float inv_rms = 1.0f / sqrtf(mean);
  // Rows whose squares leave binary32 (channels from about 2^63 on, and small ones
  // where eps is no larger) are taken times 2^-72 or 2^100, which the norm takes off again.
  const float c = ss == __builtin_inff() ? 0x1p-72f : mean < 0x1p-90f ? 0x1p100f : 1.0f;
  if (c != 1.0f) {                   // the same for the whole row
    ss = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[j][e] *= c;
        ss = __builtin_fmaf(v[j][e], v[j][e], ss);
      }
    ss = row_reduce<T, false>(ss, red[2]);
    inv_rms = 1.0f / sqrtf(ss / n + a.eps * c * c);
  }
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[j][e] *= inv_rms;
      if (a.w && tid + T * j < chunks) v[j][e] *= wr[j].get(e);
    }
  if (a.out == kRmsF32 || a.out == kRmsBf16) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int ch = tid + T * j;
      if (ch >= chunks) continue;
      const size_t at = (size_t)row * a.h + 8 * ch;
      if (a.out == kRmsF32) {
        f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.y) + at);
        p[0] = f32x4_t{v[j][0], v[j][1], v[j][2], v[j][3]};
        p[1] = f32x4_t{v[j][4], v[j][5], v[j][6], v[j][7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.y) + at) =
            u32x4_t{pack_bf16(v[j][0], v[j][1]), pack_bf16(v[j][2], v[j][3]), pack_bf16(v[j][4], v[j][5]),
                    pack_bf16(v[j][6], v[j][7])};
      }
    }
    return;
  }
  float top[CH], inv[CH], sx[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    top[j] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top[j] = nmax(top[j], tid + T * j < chunks ? fabsf(v[j][e]) : 0.0f);
  }
  if (a.out == kRmsQ8Row) {
    float m = top[0];
#pragma unroll
    for (int j = 1; j < CH; ++j) m = nmax(m, top[j]);
    m = row_reduce<T, true>(m, red[1]);
    span_scale(finite_or_nan(m), inv[0], sx[0]);
#pragma unroll
    for (int j = 1; j < CH; ++j) inv[j] = inv[0];
    if (tid == 0) a.scales[row] = sx[0];
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j) {   // h is a multiple of 32 here: lane quads are whole
      top[j] = nmax(top[j], dpp_fa<0xB1>(top[j]));
      top[j] = nmax(top[j], dpp_fa<0x4E>(top[j]));
      span_scale(finite_or_nan(top[j]), inv[j], sx[j]);
      const int ch = tid + T * j;
      if (ch < chunks && (ch & 3) == 0) a.scales[(size_t)row * (a.h >> 5) + (ch >> 2)] = sx[j];
    }
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int ch = tid + T * j;
    if (ch >= chunks) continue;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = (int)__builtin_amdgcn_fmed3f(rintf(v[j][e] * inv[j]), -127.0f, 127.0f);
      w[e >> 2] |= ((uint32_t)q & 0xffu) << (8 * (e & 3));
    }
    *reinterpret_cast<u32x2_t*>(a.codes + (size_t)row * a.h + 8 * ch) = u32x2_t{w[0], w[1]};
  }
}

template <int T, int CH>
static void launch_rms_t(const RmsNormArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)(T == 64 ? (a.rows + 3) / 4 : a.rows)), block(T < 256 ? 256 : T);
  const int kind = (a.x_f32 ? 3 : 0) + (a.res ? (a.res_f32 ? 2 : 1) : 0);
#define QG_RMS(K, X, R) \
  case K: hipLaunchKernelGGL((rms_norm_kernel<T, CH, X, R>), grid, block, 0, stream, a); break;
  switch (kind) {
    QG_RMS(0, false, 0) QG_RMS(1, false, 1) QG_RMS(2, false, 2) QG_RMS(3, true, 0) QG_RMS(4, true, 1) QG_RMS(5, true, 2)
  }
#undef QG_RMS
}

hipError_t launch_rms_norm(const RmsNormArgs& a, hipStream_t stream) {
  const int chunks = a.h >> 3;
  if (chunks <= 64)
    launch_rms_t<64, 1>(a, stream);
  else if (chunks <= 128)
    launch_rms_t<64, 2>(a, stream);
  else if (chunks <= 256)
    launch_rms_t<64, 4>(a, stream);
  else if (chunks <= 512)
    launch_rms_t<256, 2>(a, stream);
  else if (chunks <= 1024)
    launch_rms_t<256, 4>(a, stream);
  else if (chunks <= 2048)
    launch_rms_t<1024, 2>(a, stream);
  else
    launch_rms_t<1024, 4>(a, stream);
  return hipGetLastError();
}

}  // namespace qg
