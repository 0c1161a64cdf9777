// prompt_mma.cu -- attention over whole prompts in the up-projected form, on
// mma.sync.
//
// Per query row (token i, head h; q = [q_nope 128 | q_pe 64]) and key token
// j of the same sequence (k = [k_nope 128 of head h's group | k_pe 64 shared
// by all heads], value 128): out = sum_j softmax(scale * q . k_j) value_j
// over j <= i (causal) or all j.  One pass over the keys with a running
// maximum and sum per row (fp32); the weights are rounded to the I/O dtype
// for their product with the values.
//
// One CTA per 64 query rows of a head, one warp per 16 rows; key tiles of 64
// in two cp.async stages.
#include "attn.h"
#include "common.cuh"
#include "prompt_plan.cuh"

namespace mla {
namespace {

constexpr int kPrThreads = 128;
constexpr int kPrRows = 64;
constexpr int kPrKeys = 64;
constexpr int kQkD = kNope + kRope;       // 192
constexpr int kKPitch = kQkD * 2 + 16;    // 25 16-byte units
constexpr int kVPitch = kV * 2 + 16;      // 17 16-byte units
constexpr int kPrQ = 0;
constexpr int kPrK = kPrQ + kPrRows * kKPitch;
constexpr int kPrV = kPrK + 2 * kPrKeys * kKPitch;
constexpr int kPrBytes = kPrV + 2 * kPrKeys * kVPitch;

template <typename T>
__device__ __forceinline__ const T* prow(const PromptTensor& t, int b, int h, int tok) {
  return static_cast<const T*>(t.ptr) + (size_t)b * t.sb + (size_t)h * t.sh + (size_t)tok * t.st;
}

template <typename T>
__global__ void __launch_bounds__(kPrThreads) prompt_mma_kernel(const PromptParams p) {
  using E = Elem<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ PromptPlanShared plan;
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
  PromptPlace pl;
  if (!prompt_place(p, &plan, blockIdx.x, kPrRows, &pl, blockIdx.x == 0 && blockIdx.y == 0)) return;
  const int rows = min(kPrRows, pl.len - pl.row0);
  const int keys = p.causal ? pl.row0 + rows : pl.len;
  const int tiles = (keys + kPrKeys - 1) / kPrKeys;

  auto copy_row = [&](uint32_t dst, const T* src, int chunk, bool ok) { cp_async16(dst + chunk * 16, src + chunk * 8, ok ? 16 : 0); };
  // queries: 24 16-byte chunks per row
  for (int i = tid; i < kPrRows * 24; i += kPrThreads) {
    const int r = i / 24, ch = i - r * 24;
    const bool ok = r < rows;
    const int tok = pl.begin + (ok ? pl.row0 + r : 0);
    const uint32_t d = sb + kPrQ + r * kKPitch;
    if (ch < 16) copy_row(d, prow<T>(p.q_nope, pl.batch, h, tok), ch, ok);
    else copy_row(d + 256, prow<T>(p.q_pe, pl.batch, h, tok), ch - 16, ok);
  }
  auto load = [&](int tile) {
    for (int i = tid; i < kPrKeys * 40; i += kPrThreads) {
      const int r = i / 40, ch = i - r * 40;
      const bool ok = tile * kPrKeys + r < keys;
      const int tok = pl.begin + (ok ? tile * kPrKeys + r : 0);
      const uint32_t dk = sb + kPrK + ((tile & 1) * kPrKeys + r) * kKPitch;
      const uint32_t dv = sb + kPrV + ((tile & 1) * kPrKeys + r) * kVPitch;
      if (ch < 16) copy_row(dk, prow<T>(p.k_nope, pl.batch, hk, tok), ch, ok);
      else if (ch < 24) copy_row(dk + 256, prow<T>(p.k_pe, pl.batch, 0, tok), ch - 16, ok);
      else copy_row(dv, prow<T>(p.value, pl.batch, hk, tok), ch - 24, ok);
    }
  };
  load(0);
  cp_async_commit();
  float acc[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  const int r_lo = warp * 16 + (lane >> 2);
  for (int tile = 0; tile < tiles; ++tile) {
    if (tile + 1 < tiles) load(tile + 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float sc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
    const uint32_t qa = sb + kPrQ + (warp * 16 + (lane & 15)) * kKPitch + (lane >> 4) * 16;
    const uint32_t ka = sb + kPrK + ((tile & 1) * kPrKeys + (lane & 7) + ((lane >> 4) & 1) * 8) * kKPitch + ((lane >> 3) & 1) * 16;
#pragma unroll 4
    for (int k = 0; k < kQkD / 16; ++k) {
      uint32_t af[4];
      ldsm_x4(qa + k * 32, af[0], af[1], af[2], af[3]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(ka + n * 16 * kKPitch + k * 32, b0, b1, b2, b3);
        mma16816<E::kBf16>(sc[2 * n], af, b0, b1);
        mma16816<E::kBf16>(sc[2 * n + 1], af, b2, b3);
      }
    }
    // softmax: this thread holds rows r_lo and r_lo + 8, two keys of each group of 8
    float alpha[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int lim = min(keys, p.causal ? pl.row0 + r_lo + hf * 8 + 1 : keys) - tile * kPrKeys - (lane & 3) * 2;
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float& x = sc[n][2 * hf + i];
          x = n * 8 + i < lim ? x * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
      const float m_new = fmaxf(m_run[hf], mx), mu = m_new == -INFINITY ? 0.f : m_new;
      alpha[hf] = exp2f(m_run[hf] - mu);
      m_run[hf] = m_new;
      float ls = 0.f;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float& x = sc[n][2 * hf + i];
          x = exp2f(x - mu);
          ls += x;
        }
      l_run[hf] = l_run[hf] * alpha[hf] + ls;
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      acc[n][0] *= alpha[0];
      acc[n][1] *= alpha[0];
      acc[n][2] *= alpha[1];
      acc[n][3] *= alpha[1];
    }
    const uint32_t va = sb + kPrV + ((tile & 1) * kPrKeys + (lane & 15)) * kVPitch + (lane >> 4) * 16;
#pragma unroll
    for (int k = 0; k < kPrKeys / 16; ++k) {
      const uint32_t af[4] = {E::pack(sc[2 * k][0], sc[2 * k][1]), E::pack(sc[2 * k][2], sc[2 * k][3]),
                              E::pack(sc[2 * k + 1][0], sc[2 * k + 1][1]), E::pack(sc[2 * k + 1][2], sc[2 * k + 1][3])};
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_trans(va + k * 16 * kVPitch + n * 32, b0, b1, b2, b3);
        mma16816<E::kBf16>(acc[2 * n], af, b0, b1);
        mma16816<E::kBf16>(acc[2 * n + 1], af, b2, b3);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    float l = l_run[hf];
    l += __shfl_xor_sync(~0u, l, 1);
    l += __shfl_xor_sync(~0u, l, 2);
    const int r = r_lo + hf * 8;
    if (r >= rows) continue;
    const float iv = l == 0.f ? 0.f : 1.f / l;
    const int tok = pl.begin + pl.row0 + r;
    uint32_t* o = reinterpret_cast<uint32_t*>(const_cast<T*>(prow<T>(p.out, pl.batch, h, tok))) + (lane & 3);
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n * 4] = E::pack(acc[n][2 * hf] * iv, acc[n][2 * hf + 1] * iv);
    if (p.lse && (lane & 3) == 0)
      p.lse[((size_t)pl.batch * p.heads + h) * p.s + tok] = l == 0.f ? -INFINITY : (m_run[hf] + log2f(l)) * kLn2;
  }
}

template <typename T>
cudaError_t launch(const PromptParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(prompt_mma_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrBytes);
  if (e != cudaSuccess) return e;
  prompt_mma_kernel<T><<<dim3(prompt_blocks(p, kPrRows), p.heads), kPrThreads, kPrBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_mma_launch(bool bf16, const PromptParams& p, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, stream) : launch<__half>(p, stream);
}

}  // namespace mla
