// fp8_rows.cu -- rows of fp16 / bf16 to e4m3 codes with one fp32 scale per
// 128 columns of a row, after an RMSNorm or not.
//
//   y = x, or x / sqrt(mean(x^2) + eps) * gamma             (fp32)
//   s = max(max |y| / 448, 2^-126)  over the block's columns
//   code = e4m3(y * (1 / s)), to nearest even; y ~ code * s
// (s never leaves the normal range, so 1 / s is finite for every finite row;
// each step is one IEEE fp32 operation.)  The scales are stored block-major,
// [K / 128, T]: the linear layer's threads read one block's scales of
// neighbouring rows together.
//
// Two bytes in and one byte out per value, one pass: bound by memory.  A
// block of 128 columns belongs to 16 lanes, 8 values (16 bytes) each, so its
// maximum takes four shuffles.  Without a norm a lane has kUnroll blocks of
// one row in flight; with one, a row stays in registers between the sum of
// squares and the scaling: a warp's (up to 2048 columns, many rows) or a CTA's
// (up to 8192; what is beyond is read again, from L2).
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8.h"

namespace mla {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
  return v;
}

template <typename T>
__device__ __forceinline__ void to_floats(const uint4& v, float* f) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Elem<T>::to_f(e[i]);
}

// One block of 128 columns: this lane's 8 values of it, `live` where its
// columns exist.  All lanes of the warp (two blocks).
__device__ __forceinline__ void emit_block(const float* f, bool live, uint8_t* q, float* scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  m = half_warp_max(live ? m : 0.f);
  const float s = fmaxf(m / kE4m3Max, 1.17549435e-38f);  // 2^-126
  const float inv = 1.0f / s;
  if (!live) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint2*>(q) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  if ((threadIdx.x & 15) == 0) *scale = s;
}

// No norm: half-warp i of a CTA takes row 16 y + i and kUnroll blocks of
// columns, CTA = y * across + x.  (Neighbouring CTAs take neighbouring columns: 8192 x 7168 30.7
// us, 32.4 the other way round; scales gathered in shared memory first 31.5.)
template <typename T, int kUnroll>
__global__ void __launch_bounds__(kRowThreads) fp8_rows_kernel(const Fp8RowsParams p, unsigned across) {
  grid_dep_launch_dependents();
  const unsigned y = blockIdx.x / across;
  const int t = y * (kRowThreads / 16) + (threadIdx.x >> 4);
  const int kb0 = (blockIdx.x - y * across) * kUnroll, c0 = kb0 * kFp8Block + (threadIdx.x & 15) * 8;
  const T* x = static_cast<const T*>(p.x) + (long long)(t < p.T ? t : 0) * p.x_stride;
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    if (t < p.T && c0 + u * kFp8Block < p.K) v[u] = __ldcs(reinterpret_cast<const uint4*>(x + c0 + u * kFp8Block));
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int c = c0 + u * kFp8Block;
    float f[8];
    to_floats<T>(v[u], f);
    emit_block(f, t < p.T && c < p.K, p.q + (long long)t * p.q_stride + c, p.scale + (long long)(kb0 + u) * p.T + t);
  }
}

// Norm, a group of kLanes threads (a warp or the CTA) per row; the first
// kKeep vectors of a thread stay in registers.
template <typename T, int kLanes, int kKeep>
__global__ void __launch_bounds__(kRowThreads, kLanes == 32 ? 3 : 4) fp8_norm_rows_kernel(const Fp8RowsParams p) {
  grid_dep_launch_dependents();
  constexpr int kRows = kRowThreads / kLanes;
  __shared__ float part[kRowThreads / 32];
  __shared__ float scales[kRows > 1 ? kKeep * kLanes / 16 : 1][kRows];  // (a warp's rows: written together at the end)
  const int i = threadIdx.x % kLanes;
  const int t0 = blockIdx.x * kRows, t = t0 + threadIdx.x / kLanes;
  const bool row = t < p.T;  // (the same for a whole warp)
  const T* x = static_cast<const T*>(p.x) + (long long)(row ? t : 0) * p.x_stride;
  const T* gamma = static_cast<const T*>(p.gamma);
  constexpr int kStep = kLanes * 8;
  uint4 v[kKeep];
#pragma unroll
  for (int u = 0; u < kKeep; ++u) {
    const int c = u * kStep + i * 8;
    v[u] = make_uint4(0, 0, 0, 0);
    if (row && c < p.K) v[u] = *reinterpret_cast<const uint4*>(x + c);
  }
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < kKeep; ++u) {
    float f[8];
    to_floats<T>(v[u], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += f[k] * f[k];
  }
  for (int c = kKeep * kStep + i * 8; row && c < p.K; c += kStep) {
    float f[8];
    to_floats<T>(*reinterpret_cast<const uint4*>(x + c), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += f[k] * f[k];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
  if constexpr (kLanes > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) ss += part[w];
  }
  const float r = 1.0f / sqrtf(ss / (float)p.K + p.eps);
  auto block = [&](int c, const uint4& xv) {
    const uint4 gv = row && c < p.K ? __ldg(reinterpret_cast<const uint4*>(gamma + c)) : make_uint4(0, 0, 0, 0);
    float f[8], gf[8];
    to_floats<T>(xv, f);
    to_floats<T>(gv, gf);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = f[k] * r * gf[k];
    emit_block(f, row && c < p.K, p.q + (long long)t * p.q_stride + c,
               kRows > 1 ? &scales[kRows > 1 ? c / kFp8Block : 0][t - t0] : p.scale + (long long)(c / kFp8Block) * p.T + t);
  };
#pragma unroll
  for (int u = 0; u < kKeep; ++u)
    if (u * kStep < p.K) block(u * kStep + i * 8, v[u]);  // (the same for a whole warp)
  for (int c0 = kKeep * kStep; c0 < p.K; c0 += kStep) {
    const int c = c0 + i * 8;
    block(c, row && c < p.K ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0));
  }
  if constexpr (kRows > 1) {
    __syncthreads();
    for (int x = threadIdx.x; x < kKeep * kLanes / 16 * kRows; x += kRowThreads) {
      const int b = x / kRows, r = x % kRows;
      if (b * kFp8Block < p.K && t0 + r < p.T) p.scale[(long long)b * p.T + t0 + r] = scales[b][r];
    }
  }
}

template <typename T>
cudaError_t launch(const Fp8RowsParams& p, cudaStream_t stream) {
  const int blocks = (p.K + kFp8Block - 1) / kFp8Block;
  if (!p.gamma) {
    constexpr int kU = 4;
    const unsigned across = (blocks + kU - 1) / kU;
    fp8_rows_kernel<T, kU><<<(unsigned)((p.T + 15) / 16) * across, kRowThreads, 0, stream>>>(p, across);
  } else if (p.K > 2048) {
    fp8_norm_rows_kernel<T, 256, 4><<<p.T, kRowThreads, 0, stream>>>(p);
  } else if (p.T <= 1024) {  // (a CTA per row: 64 x 1536 2.1 us, 4.0 with a warp; 8192 x 1536 25.5 and 14.2)
    fp8_norm_rows_kernel<T, 256, 1><<<p.T, kRowThreads, 0, stream>>>(p);
  } else {
    const int grid = (p.T + 7) / 8;
    if (p.K <= 512)
      fp8_norm_rows_kernel<T, 32, 2><<<grid, kRowThreads, 0, stream>>>(p);
    else if (p.K <= 1024)
      fp8_norm_rows_kernel<T, 32, 4><<<grid, kRowThreads, 0, stream>>>(p);
    else if (p.K <= 1536)
      fp8_norm_rows_kernel<T, 32, 6><<<grid, kRowThreads, 0, stream>>>(p);
    else
      fp8_norm_rows_kernel<T, 32, 8><<<grid, kRowThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t fp8_rows_launch(bool bf16, const Fp8RowsParams& p, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<__half>(p, stream);
}

}  // namespace mla
