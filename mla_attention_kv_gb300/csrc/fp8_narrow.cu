// fp8_narrow.cu -- the e4m3 linear layer for few token rows:
//
//   out[t][n] = sum_b xs[b][t] * ws[n / 128][b] * sum_{k in block b} xq[t][k] wq[n][k]
//
// with blocks of 128 along K.  The weights are read once and used by few
// rows: bound by their bytes (by latency for one row).  So the weights are
// the MMA's 128-row operand and the tokens its columns (16 to 128): a tile is
// 128 weight rows, which share one weight scale per block, and its K blocks
// are split over the CTAs of a cluster, whose parts are summed through
// distributed shared memory in a fixed order (no workspace, no second
// launch).  The tensor core's sum of a block stays in tensor memory until the
// epilogue scales it and adds it to fp32 registers: one weight row and all
// tokens of the tile per thread.
//
// Warps: 0 TMA, 1 tensor memory and MMA, 2-5 epilogue.  Behind the row
// quantisation the kernel is launched early: its first weight tiles are under
// way while that one still runs.
#include <string.h>

#include "attn_tc.cuh"
#include "fp8.h"
#include "tma.h"

namespace mla {
namespace {

constexpr int kNwThreads = 192;
constexpr uint32_t kWTile = 128 * 128;

template <int TN>
struct NwCfg {
  static constexpr uint32_t kStage = kWTile + TN * 128;
  static constexpr int kStages = TN == 128 ? 3 : TN == 64 ? 4 : 5;  // two CTAs per SM
  static constexpr uint32_t kScale = kStages * kStage;             // [4 warps][2][TN] fp32
  static constexpr uint32_t kBar = kScale + 4 * 2 * TN * 4;
  static constexpr uint32_t kSmem = kBar + 256 + 1024;  // + alignment slack
  static constexpr uint32_t kTmem = 2 * TN < 32 ? 32 : 2 * TN;
  static_assert(TN * 128 * 4 <= kStages * kStage, "the sums take the stages' place");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int kStages>
struct NwShared {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort;
};

struct NwArgs {
  CUtensorMap w, x;
  Fp8LinearParams p;
};

template <typename T, int TN>
__global__ void __launch_bounds__(kNwThreads, 2) fp8_narrow_kernel(const __grid_constant__ NwArgs a) {
  using E = Elem<T>;
  using S = NwCfg<TN>;
  const Fp8LinearParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  using Sh = NwShared<S::kStages>;
  static_assert(sizeof(Sh) <= 256, "barrier block");
  Sh* sh = reinterpret_cast<Sh*>(smem + S::kBar);
  const uint32_t sbase = smem_u32(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };
  const int split = gridDim.x, rank = blockIdx.x;  // (a cluster is a row of the grid)
  const int nt = blockIdx.y, t0 = blockIdx.z * TN;
  const int blocks = (p.K + kFp8Block - 1) / kFp8Block;
  const int b0 = (int)((long long)blocks * rank / split), nb = (int)((long long)blocks * (rank + 1) / split) - b0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(bar(&sh->full[i]), 1);
      mbar_init(bar(&sh->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh->tfull[i]), 1);
      mbar_init(bar(&sh->tempty[i]), 4);
    }
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(smem_u32(&sh->tmem), S::kTmem);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  float2 acc[TN / 2];  // (epilogue warps)
  if (warp == 0) {
    // ============================================================ TMA
    if (lane == 0) {
      const int ahead = min(nb, S::kStages);
      for (int i = 0; i < ahead; ++i) {  // weights first: they do not depend on the kernel before
        mbar_arrive_expect_tx(bar(&sh->full[i]), S::kStage);
        tma_load_2d(sbase + i * S::kStage, &a.w, (b0 + i) * kFp8Block, nt * 128, bar(&sh->full[i]));
      }
      grid_dep_wait();
      for (int i = 0; i < ahead; ++i)
        tma_load_2d(sbase + i * S::kStage + kWTile, &a.x, (b0 + i) * kFp8Block, t0, bar(&sh->full[i]));
      int fills = ahead;
      for (int i = ahead; i < nb; ++i) {
        const int st = i % S::kStages;
        if (!at_wait(bar(&sh->empty[st]), ((i / S::kStages) & 1) ^ 1, abort, p.budget_ns, p.status)) break;
        mbar_arrive_expect_tx(bar(&sh->full[st]), S::kStage);
        tma_load_2d(sbase + st * S::kStage, &a.w, (b0 + i) * kFp8Block, nt * 128, bar(&sh->full[st]));
        tma_load_2d(sbase + st * S::kStage + kWTile, &a.x, (b0 + i) * kFp8Block, t0, bar(&sh->full[st]));
        ++fills;
      }
      for (int i = 0; i < S::kStages; ++i) {  // every copy has landed before the CTA may go on
        const uint32_t n = ring_uses(fills, S::kStages, i);
        if (n > 0) mbar_wait_bounded(bar(&sh->full[i]), (n - 1) & 1, drain_budget(p.budget_ns));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ MMA
    if (tc::elect_one()) {
      constexpr uint32_t idesc = tc::idesc_e4m3(128, TN);
      const uint64_t dw = tc::sdesc_sw128(sbase, 16, 1024), dx = tc::sdesc_sw128(sbase + kWTile, 16, 1024);
      for (int i = 0; i < nb; ++i) {
        const int st = i % S::kStages, buf = i & 1;
        if (!(i == 0 ? at_wait_poll(bar(&sh->full[st]), 0, abort, p.budget_ns, p.status)
                     : at_wait(bar(&sh->full[st]), (i / S::kStages) & 1, abort, p.budget_ns, p.status)))
          break;
        if (!at_wait(bar(&sh->tempty[buf]), ((i >> 1) & 1) ^ 1, abort, p.budget_ns, p.status)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma_f8(tmem + buf * TN, dw + st * (S::kStage >> 4) + 2 * k, dx + st * (S::kStage >> 4) + 2 * k, idesc, k > 0);
        tc::commit(bar(&sh->empty[st]));
        tc::commit(bar(&sh->tfull[buf]));
      }
      tc::commit(bar(&sh->done));
      mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));
    }
    __syncwarp();
  } else {
    // ============================================================ epilogue: scaled sums
    const int e = warp - 2;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* sc = reinterpret_cast<float*>(smem + S::kScale) + e * 2 * TN;
    constexpr int kMine = (TN + 31) / 32;
#pragma unroll
    for (int j = 0; j < TN / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    grid_dep_wait();
    auto scales = [&](int i, float* s) {  // of K block b0 + i: this lane's tokens
      const float w = i < nb ? __ldg(p.w_scale + (size_t)nt * blocks + b0 + i) : 0.f;
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int t = t0 + u * 32 + lane;
        s[u] = i < nb && (TN >= 32 || lane < TN) && t < p.T ? w * __ldg(p.x_scale + (size_t)(b0 + i) * p.T + t) : 0.f;
      }
    };
    float next[kMine];
    scales(0, next);
    for (int i = 0; i < nb; ++i) {
      const int buf = i & 1;
      float* s = sc + buf * TN;
#pragma unroll
      for (int u = 0; u < kMine; ++u)
        if (TN >= 32 || lane < TN) s[u * 32 + lane] = next[u];
      scales(i + 1, next);
      __syncwarp();
      if (!at_wait_warp(bar(&sh->tfull[buf]), (i >> 1) & 1, abort, p.budget_ns, p.status)) break;
      tc::fence_after_sync();
      constexpr int kCols = TN < 32 ? 16 : 32;
#pragma unroll
      for (int c = 0; c < TN; c += kCols) {
        uint32_t v[kCols];
        if constexpr (kCols == 16)
          tc::ld16(tl + buf * TN + c, v);
        else
          tc::ld32(tl + buf * TN + c, v);
        tc::wait_ld();
        if (c + kCols == TN) {  // the last columns are in registers
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&sh->tempty[buf]));
        }
#pragma unroll
        for (int k = 0; k < kCols; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s + c + k);
          float2* d = acc + (c + k) / 2;
          d[0].x = fmaf(__uint_as_float(v[k]), f.x, d[0].x);
          d[0].y = fmaf(__uint_as_float(v[k + 1]), f.y, d[0].y);
          d[1].x = fmaf(__uint_as_float(v[k + 2]), f.z, d[1].x);
          d[1].y = fmaf(__uint_as_float(v[k + 3]), f.w, d[1].y);
        }
      }
    }
  }

  // ---- sums over the cluster: [token][weight row] in the stages' place
  __syncthreads();  // (all MMAs and copies are through)
  if (warp >= 2) {
    float* red = reinterpret_cast<float*>(smem) + (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < TN / 2; ++j) {
      red[(2 * j) * 128] = acc[j].x;
      red[(2 * j + 1) * 128] = acc[j].y;
    }
  }
  if (split > 1) tc::cluster_sync(); else __syncthreads();
  if (warp >= 2) {
    const int live = min(TN, p.T - t0);
    const int n = nt * 128 + lane * 4;
    for (int j = live * rank / split + warp - 2; j < live * (rank + 1) / split; j += 4) {
      const uint32_t at = sbase + (j * 128 + lane * 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < split; ++r) {
        float4 v;
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(tc::mapa(at, r))
                     : "memory");
        y.x += v.x;
        y.y += v.y;
        y.z += v.z;
        y.w += v.w;
      }
      if (n < p.N)  // (N is a multiple of 8)
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (size_t)(t0 + j) * p.out_stride + n) =
            make_uint2(E::pack(y.x, y.y), E::pack(y.z, y.w));
    }
  }
  if (split > 1) tc::cluster_sync();  // (no CTA leaves while another reads its sums)
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, S::kTmem);
  }
}

template <typename T, int TN>
cudaError_t launch(const Fp8LinearParams& p, const Fp8Maps& maps, int num_sms, cudaStream_t stream) {
  NwArgs a;
  a.w = maps.w; a.x = maps.x; a.p = p;
  const int blocks = (p.K + kFp8Block - 1) / kFp8Block, nt = (p.N + 127) / 128, tt = (p.T + TN - 1) / TN;
  int split = 1;
  while (split < 8 && 2 * split <= blocks && (long long)nt * tt * split * 2 <= 2 * num_sms) split *= 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(split, nt, tt);
  c.blockDim = dim3(kNwThreads);
  c.dynamicSmemBytes = NwCfg<TN>::kSmem;
  c.stream = stream;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = p.dependent ? 2 : 1;
  return cudaLaunchKernelEx(&c, fp8_narrow_kernel<T, TN>, a);
}

template <typename T>
cudaError_t launch_tn(const Fp8LinearParams& p, const void* xq, int xq_stride, Fp8Maps* maps, int num_sms, cudaStream_t stream) {
  const int tn = p.T <= 16 ? 16 : p.T <= 32 ? 32 : p.T <= 64 ? 64 : 128;
  if (!fp8_row_map(maps, xq, p.T, p.K, xq_stride, tn)) return cudaErrorInvalidValue;
  switch (tn) {
    case 16: return launch<T, 16>(p, *maps, num_sms, stream);
    case 32: return launch<T, 32>(p, *maps, num_sms, stream);
    case 64: return launch<T, 64>(p, *maps, num_sms, stream);
    default: return launch<T, 128>(p, *maps, num_sms, stream);
  }
}

template <typename T, int TN>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(fp8_narrow_kernel<T, TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, NwCfg<TN>::kSmem);
}
template <typename T>
cudaError_t prepare() {
  cudaError_t e = prepare_one<T, 16>();
  if (e == cudaSuccess) e = prepare_one<T, 32>();
  if (e == cudaSuccess) e = prepare_one<T, 64>();
  if (e == cudaSuccess) e = prepare_one<T, 128>();
  return e;
}

}  // namespace

bool fp8_row_map(Fp8Maps* maps, const void* xq, int T, int K, int stride, int box) {
  Fp8Maps::Key key;
  memset(&key, 0, sizeof(key));
  key.x = xq; key.T = T; key.stride = stride; key.box = box;
  if (maps->valid && memcmp(&key, &maps->key, sizeof(key)) == 0) return true;
  maps->valid = false;
  if (!encode_tmap_2d(&maps->x, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)K, (uint64_t)T, (uint64_t)stride, kFp8Block, (uint32_t)box,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return false;
  maps->key = key;
  maps->valid = true;
  return true;
}

cudaError_t fp8_narrow_prepare() {
  const cudaError_t e = prepare<__half>();
  return e == cudaSuccess ? prepare<__nv_bfloat16>() : e;
}

cudaError_t fp8_narrow_launch(bool bf16, const Fp8LinearParams& p, const void* xq, int xq_stride, Fp8Maps* maps, int num_sms,
                              cudaStream_t stream) {
  return bf16 ? launch_tn<__nv_bfloat16>(p, xq, xq_stride, maps, num_sms, stream)
              : launch_tn<__half>(p, xq, xq_stride, maps, num_sms, stream);
}

}  // namespace mla
