// fp8_pair.cu -- the e4m3 linear layer for many token rows (formula in
// fp8_narrow.cu), on the 2-SM tensor-core MMA: a pair of CTAs takes tiles of
// 256 token rows x 256 weight rows, each CTA loading its 128 rows of either
// operand by TMA.
//
// The scales change with every block of 128 along K, so the tensor core's
// sums cannot run on: a block's sums (4 MMAs of K = 32, 512 cycles) go to one
// of two halves of tensor memory, and the epilogue warps take them from
// there, scale them and add them to fp32 registers while the next block's
// MMAs run.  Eight epilogue warps per CTA, a thread holding one token row and
// the 128 columns of one weight block, so that the two scales are one factor
// per thread and block: 128 FMAs (as 64 packed ones) on 128 registers.
//
// Warps: 0 TMA, 1 tensor memory and (even CTA) MMA, 2-9 epilogue.
#include <string.h>

#include "attn_tc.cuh"
#include "fp8.h"
#include "tma.h"

namespace mla {
namespace {

constexpr int kPrThreads = 320;
constexpr int kPrEpi = 8;
constexpr uint32_t kPrStage = 32768;  // this CTA's 128 token rows and 128 weight rows of a K block
constexpr int kPrStages = 6;
constexpr uint32_t kPrBar = kPrStages * kPrStage;
constexpr uint32_t kPrOut = kPrBar + 512;  // per epilogue warp 32 rows x 128 bytes of results
constexpr uint32_t kPrSmem = kPrOut + kPrEpi * 4096 + 1024;  // + alignment slack
static_assert(kPrSmem <= 227 * 1024, "shared memory");

struct PrShared {
  uint64_t full[kPrStages], empty[kPrStages], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PrShared) <= 512, "barrier block");

struct PrArgs {
  CUtensorMap w, x;
  Fp8LinearParams p;
  int nm, nn, m_fast;
};

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrThreads, 1) fp8_pair_kernel(const __grid_constant__ PrArgs a) {
  using E = Elem<T>;
  const Fp8LinearParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  PrShared* sh = reinterpret_cast<PrShared*>(smem + kPrBar);
  const uint32_t sbase = smem_u32(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };
  auto lead = [](uint64_t* b) { return tc::mapa(smem_u32(b), 0); };
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int blocks = (p.K + kFp8Block - 1) / kFp8Block, tiles = a.nm * a.nn;
  // tile u: token tiles or weight tiles fastest
  auto tile_m = [&](int u) { return a.m_fast ? u % a.nm : u / a.nn; };
  auto tile_n = [&](int u) { return a.m_fast ? u / a.nm : u % a.nn; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPrStages; ++i) {
      mbar_init(bar(&sh->full[i]), 1);
      mbar_init(bar(&sh->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh->tfull[i]), 1);
      mbar_init(bar(&sh->tempty[i]), 2 * kPrEpi);
    }
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc2(smem_u32(&sh->tmem), 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers are initialised before any copy, commit or arrival reaches them
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  if (warp == 0) {
    // ============================================================ TMA
    if (lane == 0) {
      grid_dep_wait();
      uint32_t s = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += pairs) {
        const int m0 = tile_m(u) * 256 + rank * 128, n0 = tile_n(u) * 256 + rank * 128;
        for (int b = 0; b < blocks; ++b) {
          const uint32_t st = s % kPrStages;
          ok = at_wait(bar(&sh->empty[st]), ((s / kPrStages) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          const uint32_t dst = sbase + st * kPrStage, fb = lead(&sh->full[st]);
          if (rank == 0) mbar_arrive_expect_tx(bar(&sh->full[st]), 2 * kPrStage);
          tma_load_2d_pair(dst, &a.x, b * kFp8Block, m0, fb);
          tma_load_2d_pair(dst + 16384, &a.w, b * kFp8Block, n0, fb);
          ++s;
        }
      }
      // Every copy has landed, and every release of a slot has arrived, before the CTAs may exit.  After a wait that ran
      // out the two CTAs may have filled different numbers of slots: a fill that the other CTA has not matched is never
      // released, and its waits take the whole limit, in which it lands.
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint64_t* b, uint32_t par) {
        const uint64_t spent = globaltimer_ns() - t0, limit = drain_budget(p.budget_ns);
        mbar_wait_bounded(bar(b), par, spent < limit ? limit - spent : 0);
      };
      for (int i = 0; i < kPrStages; ++i) {
        const uint32_t n = ring_uses(s, kPrStages, i);
        if (n == 0) break;
        if (rank == 0) drain(&sh->full[i], (n - 1) & 1);
        drain(&sh->empty[i], (n - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ MMA (one thread of the even CTA)
    if (rank == 0 && tc::elect_one()) {
      constexpr uint32_t idesc = tc::idesc_e4m3(256, 256);
      const uint64_t dx = tc::sdesc_sw128(sbase, 16, 1024), dw = tc::sdesc_sw128(sbase + 16384, 16, 1024);
      uint32_t s = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += pairs) {
#pragma unroll 1
        for (int b = 0; b < blocks; ++b, ++s) {
          const uint32_t st = s % kPrStages, buf = s & 1;
          ok = (s == 0 ? at_wait_poll(bar(&sh->full[st]), 0, abort, p.budget_ns, p.status)
                       : at_wait(bar(&sh->full[st]), (s / kPrStages) & 1, abort, p.budget_ns, p.status)) &&
               at_wait<true>(bar(&sh->tempty[buf]), ((s >> 1) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma2_f8(tmem + buf * 256, dx + st * (kPrStage >> 4) + 2 * k, dw + st * (kPrStage >> 4) + 2 * k, idesc, k > 0);
          tc::commit2_both(bar(&sh->empty[st]));
          tc::commit2_both(bar(&sh->tfull[buf]));
        }
      }
      tc::commit2_both(bar(&sh->done));
    }
    __syncwarp();
  } else {
    // ============================================================ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
    unsigned char* stg = smem + kPrOut + (warp - 2) * 4096;
    uint32_t s = 0;
    bool ok = true;
    grid_dep_wait();
    for (int u = pair; u < tiles && ok; u += pairs) {
      const int row0 = tile_m(u) * 256 + rank * 128 + q * 32, t = row0 + lane;
      const int nblk = tile_n(u) * 2 + half;
      const bool live = t < p.T && nblk * 128 < p.N;
      const float* xs = p.x_scale + (live ? t : 0);
      const float* ws = p.w_scale + (live ? (size_t)nblk * blocks : 0);
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      float fx = __ldg(xs), fw = __ldg(ws);
#pragma unroll 1
      for (int b = 0; b < blocks; ++b, ++s) {
        const uint32_t buf = s & 1;
        const float f = fx * fw;
        if (b + 1 < blocks) {
          fx = __ldg(xs + (size_t)(b + 1) * p.T);
          fw = __ldg(ws + b + 1);
        }
        const uint64_t f2 = f2_pack(f, f);
        ok = at_wait_warp(bar(&sh->tfull[buf]), (s >> 1) & 1, abort, p.budget_ns, p.status);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[32];
          tc::ld32(tl + buf * 256 + c, v);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[c / 2 + i] = f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, acc[c / 2 + i]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::arrive_cluster_relaxed(lead(&sh->tempty[buf]));
      }
      if (!ok) break;
      // ---- results, 64 columns at a time: a lane writes its row's 128 bytes (16-byte units swizzled by the row), then a
      // store instruction takes 128 bytes of four rows
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col0 = nblk * 128 + h * 64;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y0, y1;
            f2_unpack(acc[h * 32 + k * 4 + i], y0, y1);
            o[i] = E::pack(y0, y1);
          }
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int c = col0 + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          if (row0 + r < p.T && c < p.N)  // (N is a multiple of 8)
            *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)(row0 + r) * p.out_stride + c) =
                *reinterpret_cast<const uint4*>(stg + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
        __syncwarp();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));  // every MMA issued has completed
  // neither CTA leaves, or releases the pair's tensor memory, while its peer may still copy into it, read it, or arrive
  // on its barriers
  tc::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

template <typename T>
cudaError_t launch(const Fp8LinearParams& p, const Fp8Maps& maps, int num_sms, cudaStream_t stream) {
  PrArgs a;
  a.w = maps.w; a.x = maps.x; a.p = p;
  a.nm = (p.T + 255) / 256;
  a.nn = (p.N + 255) / 256;
  // the operand that is smaller stays in L2 while the other streams past it
  a.m_fast = (long long)p.T < (long long)p.N;
  const long long tiles = (long long)a.nm * a.nn;
  const int pairs = tiles < num_sms / 2 ? (int)tiles : num_sms / 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(pairs * 2);
  c.blockDim = dim3(kPrThreads);
  c.dynamicSmemBytes = kPrSmem;
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = p.dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, fp8_pair_kernel<T>, a);
}

}  // namespace

cudaError_t fp8_pair_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(fp8_pair_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem);
  return e == cudaSuccess ? cudaFuncSetAttribute(fp8_pair_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem) : e;
}

cudaError_t fp8_pair_launch(bool bf16, const Fp8LinearParams& p, const void* xq, int xq_stride, Fp8Maps* maps, int num_sms,
                            cudaStream_t stream) {
  if (!fp8_row_map(maps, xq, p.T, p.K, xq_stride, 128)) return cudaErrorInvalidValue;
  return bf16 ? launch<__nv_bfloat16>(p, *maps, num_sms, stream) : launch<__half>(p, *maps, num_sms, stream);
}

}  // namespace mla
