// append.cu -- latent cache append: RMSNorm of the compressed rows, RoPE of
// the key (and query) position parts, scatter into the paged latent cache.
//
//   n = x / sqrt(mean(x^2) + eps) * gamma          (512 columns, fp32)
//   r[j]      = y[2j]   * cos[j]      - y[2j+1] * sin[j]        (j < 32)
//   r[32 + j] = y[2j+1] * cos[32 + j] + y[2j]   * sin[32 + j]
//
// Every row is read and written once (a row of x stays in registers between
// the sum of squares and the scaling), each value rounded once to the I/O
// dtype.  Bound by memory traffic for many rows and by one launch for a
// decode step.  Two kinds of blocks share the launch: key blocks (one warp
// per token row) and query blocks (eight lanes per (token, head), 16 bytes a
// lane, four heads in flight).  The queries pass through once, so they are
// read and written with the streaming hint: 16384 rows of 128 heads, 583 MB,
// take 106 us with it (5.5 TB/s) and 114 us without.
#include "attn.h"
#include "common.cuh"

namespace mla {
namespace {

constexpr int kApThreads = 256;
constexpr int kApRows = kApThreads / 32;       // key rows per block
constexpr int kApUnroll = 4;
constexpr int kApUnits = kApThreads / 8 * kApUnroll;  // (token, head) pairs per query block

__device__ __forceinline__ int append_pos(const AppendParams& p, int t) {
  int pos = p.positions[t];
  if (pos < 0 || pos >= p.max_pos) {
    atomicOr(p.status, kStatusBadPosition);
    pos = pos < 0 ? 0 : p.max_pos - 1;
  }
  return pos;
}

template <typename T>
__global__ void __launch_bounds__(kApThreads) append_kernel(const AppendParams p, int key_blocks) {
  using E = Elem<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < key_blocks) {
    const int t = blockIdx.x * kApRows + warp;
    if (t >= p.T) return;
    const int slot = p.slots[t];
    if (slot < 0) return;
    if (slot >= p.nslots) {
      if (lane == 0) atomicOr(p.status, kStatusBadSlot);
      return;
    }
    const uint4* x4 = reinterpret_cast<const uint4*>(static_cast<const T*>(p.ckv) + (size_t)t * p.ckv_stride);
    const uint4 a = x4[lane], b = x4[lane + 32];
    // (two 16-bit values per lane: the pair the rotation mixes)
    const uint32_t yy = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.kpe) + (size_t)t * p.kpe_stride)[lane];
    uint4 o[2] = {a, b};
    if (p.gamma) {
      const uint4* g4 = static_cast<const uint4*>(p.gamma);
      const uint4 g[2] = {g4[lane], g4[lane + 32]};
      const T* xe = reinterpret_cast<const T*>(o);
      const T* ge = reinterpret_cast<const T*>(g);
      float v[16], ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = E::to_f(xe[i]);
        ss += v[i] * v[i];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
      const float r = 1.0f / sqrtf(ss * (1.0f / kRank) + p.eps);
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = E::pack(v[2 * i] * r * E::to_f(ge[2 * i]), v[2 * i + 1] * r * E::to_f(ge[2 * i + 1]));
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    uint4* d4 = reinterpret_cast<uint4*>(static_cast<T*>(p.latent_cache) + (size_t)slot * p.lat_rs);
    d4[lane] = o[0];
    d4[lane + 32] = o[1];
    uint32_t* dk = reinterpret_cast<uint32_t*>(static_cast<T*>(p.kpe_cache) + (size_t)slot * p.kpe_rs);
    if (!p.cos_t) {
      dk[lane] = yy;
      return;
    }
    const int pos = append_pos(p, t);
    const float* c = p.cos_t + (size_t)pos * kRope;
    const float* s = p.sin_t + (size_t)pos * kRope;
    const T* ye = reinterpret_cast<const T*>(&yy);
    const float y0 = E::to_f(ye[0]), y1 = E::to_f(ye[1]);
    const float lo = y0 * c[lane] - y1 * s[lane];
    const float hi = y1 * c[lane + 32] + y0 * s[lane + 32];
    // lanes 0-15 store outputs 2l, 2l + 1; lanes 16-31 the same of the upper half
    const int from = 2 * (lane & 15);
    const float l0 = __shfl_sync(~0u, lo, from), l1 = __shfl_sync(~0u, lo, from + 1);
    const float h0 = __shfl_sync(~0u, hi, from), h1 = __shfl_sync(~0u, hi, from + 1);
    dk[lane] = lane < 16 ? E::pack(l0, l1) : E::pack(h0, h1);
    return;
  }
  // query heads: eight lanes per (token, head); lane i turns pairs 4i .. 4i+3
  const int i = threadIdx.x & 7;
  const long long u0 = (long long)(blockIdx.x - key_blocks) * kApUnits + (threadIdx.x >> 3);
  const long long units = (long long)p.T * p.heads;
  uint4 x[kApUnroll];
  int tt[kApUnroll], hh[kApUnroll];
#pragma unroll
  for (int k = 0; k < kApUnroll; ++k) {
    const long long u = u0 + k * (kApThreads / 8);
    tt[k] = -1;
    hh[k] = 0;
    if (u < units) {
      tt[k] = (int)(u / p.heads);
      hh[k] = (int)(u - (long long)tt[k] * p.heads);
      x[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.qpe) + (size_t)tt[k] * p.q_ts + (size_t)hh[k] * p.q_hs) + i);
    }
  }
  __syncwarp();  // in place: all of a row is read before any of it is written
#pragma unroll
  for (int k = 0; k < kApUnroll; ++k) {
    if (tt[k] < 0) continue;
    uint2* d = reinterpret_cast<uint2*>(static_cast<T*>(p.qpe_out) + (size_t)tt[k] * p.qo_ts + (size_t)hh[k] * p.qo_hs);
    const int pos = append_pos(p, tt[k]);
    const float4* c4 = reinterpret_cast<const float4*>(p.cos_t + (size_t)pos * kRope);
    const float4* s4 = reinterpret_cast<const float4*>(p.sin_t + (size_t)pos * kRope);
    const float4 cl = __ldg(c4 + i), ch = __ldg(c4 + i + 8), sl = __ldg(s4 + i), sh = __ldg(s4 + i + 8);
    const T* xe = reinterpret_cast<const T*>(&x[k]);
    float e[4], f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[j] = E::to_f(xe[2 * j]);
      f[j] = E::to_f(xe[2 * j + 1]);
    }
    __stcs(d + i, make_uint2(E::pack(e[0] * cl.x - f[0] * sl.x, e[1] * cl.y - f[1] * sl.y),
                      E::pack(e[2] * cl.z - f[2] * sl.z, e[3] * cl.w - f[3] * sl.w)));
    __stcs(d + i + 8, make_uint2(E::pack(f[0] * ch.x + e[0] * sh.x, f[1] * ch.y + e[1] * sh.y),
                          E::pack(f[2] * ch.z + e[2] * sh.z, f[3] * ch.w + e[3] * sh.w)));
  }
}

}  // namespace

cudaError_t append_launch(bool bf16, const AppendParams& p, cudaStream_t stream) {
  const int kb = (p.T + kApRows - 1) / kApRows;
  const long long qb = p.qpe ? ((long long)p.T * p.heads + kApUnits - 1) / kApUnits : 0;
  const unsigned grid = (unsigned)(kb + qb);
  if (bf16)
    append_kernel<__nv_bfloat16><<<grid, kApThreads, 0, stream>>>(p, kb);
  else
    append_kernel<__half><<<grid, kApThreads, 0, stream>>>(p, kb);
  return cudaGetLastError();
}

}  // namespace mla
