// fp8_wide.cu -- the e4m3 linear layer for many token rows (formula in
// fp8_narrow.cu): persistent CTAs on tiles of 128 token rows x 256 weight
// rows.
//
// The scales change with every block of 128 along K, so the tensor core's
// sums cannot run on: a block's sums go to tensor memory, and the epilogue
// warps take them from there, scale them and add them to fp32 registers while
// the next block's MMAs run.  A block of a tile is two MMA groups of 128
// weight rows (one weight scale each, 256 cycles); tensor memory holds four
// such results.  Sixteen epilogue warps: a thread holds one token row and 64
// columns of one weight block.  With eight, which hold twice as much, the way
// of a warp through a block (wait, load, scale, release) is the bound: 1024 x
// 16384 -> 7168 takes 152 us instead of 123.
//
// 8192 x 1536 -> 24576: 241 us (2560 TFLOP/s); without the epilogue, loads and
// MMAs alone take 231 on a ring of three stages (209 on four, whose room the
// results' staging takes).  The CTAs do not pair up for the 2-SM MMA, which
// halves the weight traffic (loads and MMAs alone 151 us) but sends commits
// and releases across the pair, about 1000 cycles a way.  Pairs took 296 us with
// eight epilogue warps that store their results themselves; single CTAs took 288 with
// sixteen such warps.  Pairs with sixteen and results by TMA were not measured.
//
// Warps: 0 TMA, 1 tensor memory, 1 and 2 MMA, 4-19 epilogue (3 only gives its
// registers).
#include "attn_tc.cuh"
#include "fp8.h"
#include "tma.h"

namespace mla {
namespace {

constexpr int kWdThreads = 640;
constexpr int kWdEpi = 16;
constexpr uint32_t kWdStage = 49152;  // 128 token rows and 256 weight rows of a K block
constexpr int kWdStages = 3;
constexpr uint32_t kWdOut = kWdStages * kWdStage;  // per epilogue warp 32 rows x 128 bytes of results
constexpr uint32_t kWdBar = kWdOut + kWdEpi * 4096;
constexpr uint32_t kWdSmem = kWdBar + 512 + 1024;  // + alignment slack
static_assert(kWdSmem <= 227 * 1024, "shared memory");
constexpr int kWdBufs = 4;  // of 128 tensor memory columns
// Registers: 640 threads are launched with 96 each; the first four warps give
// theirs up to the sixteen epilogue warps (128 * 32 + 512 * 112 = 640 * 96).
constexpr int kWdRoleRegs = 32, kWdEpiRegs = 112;

struct WdShared {
  uint64_t full[kWdStages], empty[kWdStages], tfull[kWdBufs], tempty[kWdBufs], done[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(WdShared) <= 512, "barrier block");

struct WdArgs {
  CUtensorMap w, x, out;
  Fp8LinearParams p;
  int nm, nn, group;
};

template <typename T>
__global__ void __launch_bounds__(kWdThreads, 1) fp8_wide_kernel(const __grid_constant__ WdArgs a) {
  using E = Elem<T>;
  const Fp8LinearParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  WdShared* sh = reinterpret_cast<WdShared*>(smem + kWdBar);
  const uint32_t sbase = smem_u32(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };
  const int blocks = (p.K + kFp8Block - 1) / kFp8Block, tiles = a.nm * a.nn;
  // tile u: groups of token tiles in turn; within a group, its token tiles fastest
  auto tile_at = [&](int u, int& m, int& n) {
    const int per = a.group * a.nn, g = u / per, r = u - g * per, w = min(a.group, a.nm - g * a.group);
    n = r / w;
    m = g * a.group + r - n * w;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWdStages; ++i) {
      mbar_init(bar(&sh->full[i]), 1);
      mbar_init(bar(&sh->empty[i]), 2);  // both MMA warps
    }
    for (int i = 0; i < kWdBufs; ++i) {
      mbar_init(bar(&sh->tfull[i]), 1);
      mbar_init(bar(&sh->tempty[i]), kWdEpi / 2);
    }
    for (int i = 0; i < 2; ++i) mbar_init(bar(&sh->done[i]), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(smem_u32(&sh->tmem), 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWdRoleRegs));
  if (warp == 0) {
    // ============================================================ TMA
    if (lane == 0) {
      grid_dep_wait();
      uint32_t s = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < tiles && ok; u += gridDim.x) {
        int m0, n0;
        tile_at(u, m0, n0);
        m0 *= 128;
        n0 *= 256;
        for (int b = 0; b < blocks; ++b, ++s) {
          const uint32_t st = s % kWdStages;
          ok = at_wait(bar(&sh->empty[st]), ((s / kWdStages) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          const uint32_t dst = sbase + st * kWdStage, fb = bar(&sh->full[st]);
          mbar_arrive_expect_tx(fb, kWdStage);
          tma_load_2d(dst, &a.x, b * kFp8Block, m0, fb);
          tma_load_2d(dst + 16384, &a.w, b * kFp8Block, n0, fb);
          tma_load_2d(dst + 32768, &a.w, b * kFp8Block, n0 + 128, fb);
        }
      }
      for (int i = 0; i < kWdStages; ++i) {  // every copy has landed before the CTA may exit
        const uint32_t n = ring_uses(s, kWdStages, i);
        if (n > 0) mbar_wait_bounded(bar(&sh->full[i]), (n - 1) & 1, drain_budget(p.budget_ns));
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ============================================================ MMA: a warp for each weight block of the tile
    if (tc::elect_one()) {
      const int h = warp - 1;
      constexpr uint32_t idesc = tc::idesc_e4m3(128, 128);
      const uint64_t dx = tc::sdesc_sw128(sbase, 16, 1024), dw = tc::sdesc_sw128(sbase + 16384 + h * 16384, 16, 1024);
      uint32_t s = 0, st = 0, par = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < tiles && ok; u += gridDim.x) {
#pragma unroll 1
        for (int b = 0; b < blocks; ++b, ++s) {
          const uint32_t buf = (s & 1) * 2 + h;
          ok = (s == 0 ? at_wait_poll(bar(&sh->full[st]), 0, abort, p.budget_ns, p.status)
                       : at_wait(bar(&sh->full[st]), par, abort, p.budget_ns, p.status)) &&
               at_wait(bar(&sh->tempty[buf]), ((s >> 1) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f8(tmem + buf * 128, dx + st * (kWdStage >> 4) + 2 * k, dw + st * (kWdStage >> 4) + 2 * k, idesc, k > 0);
          tc::commit(bar(&sh->tfull[buf]));
          tc::commit(bar(&sh->empty[st]));
          if (++st == kWdStages) st = 0, par ^= 1;
        }
      }
      tc::commit(bar(&sh->done[h]));
      mbar_wait_bounded(bar(&sh->done[h]), 0, drain_budget(p.budget_ns));  // every MMA issued has completed
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ============================================================ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWdEpiRegs));
    const int q = warp & 3, e = (warp - 4) >> 2;  // lanes
    const int h = e >> 1, g = e & 1;              // weight block of the tile, half of its columns
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + h * 128 + g * 64;
    const uint32_t full[2] = {bar(&sh->tfull[h]), bar(&sh->tfull[2 + h])}, empty[2] = {bar(&sh->tempty[h]), bar(&sh->tempty[2 + h])};
    const uint32_t out = kWdOut + (warp - 4) * 4096;
    uint32_t s = 0;
    bool ok = true;
    grid_dep_wait();
    for (int u = blockIdx.x; u < tiles && ok; u += gridDim.x) {
      int tm, tn;
      tile_at(u, tm, tn);
      const int row0 = tm * 128 + q * 32, t = row0 + lane, nblk = tn * 2 + h;
      const float* xs = p.x_scale + (t < p.T ? t : 0);
      const float* ws = p.w_scale + (nblk * 128 < p.N ? (size_t)nblk * blocks : 0);
      uint64_t acc[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[i] = 0;
      float fx = ld_behind_dep(xs), fw = __ldg(ws);
#pragma unroll 1
      for (int b = 0; b < blocks; ++b, ++s) {
        const float f = fx * fw;
        if (b + 1 < blocks) {
          xs += p.T;
          fx = ld_behind_dep(xs);
          fw = __ldg(ws + b + 1);
        }
        const uint64_t f2 = f2_pack(f, f);
        const uint32_t tb = tl + (s & 1) * 256;
        if (!__all_sync(~0u, mbar_try_wait(s & 1 ? full[1] : full[0], (s >> 1) & 1)))
          ok = at_wait_warp(s & 1 ? full[1] : full[0], (s >> 1) & 1, abort, p.budget_ns, p.status);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t v[32];
        tc::ld32(tb, v);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[i] = f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, acc[i]);
        tc::ld32(tb + 32, v);
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s & 1 ? empty[1] : empty[0]);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[16 + i] = f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, acc[16 + i]);
      }
      if (!ok) break;
      // ---- results: a lane writes its row's 128 bytes (16-byte units swizzled by the row), and one copy takes the warp's
      // 32 rows to memory while the next tile is under way (rows past T and columns past N are left out by the map)
      if (lane == 0) bulk_wait_read();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y0, y1;
          f2_unpack(acc[k * 4 + i], y0, y1);
          o[i] = E::pack(y0, y1);
        }
        *reinterpret_cast<uint4*>(smem + out + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      const int c = nblk * 128 + g * 64;
      if (lane == 0 && row0 < p.T && c < p.N) {
        tma_store_2d(&a.out, sbase + out, c, row0);
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait_all();  // (shared memory is read until then)
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <typename T>
cudaError_t launch(const Fp8LinearParams& p, const CUtensorMap& w, const void* xq, int xq_stride, int num_sms, cudaStream_t stream) {
  WdArgs a;
  a.w = w; a.p = p;
  // (results in boxes of 32 rows x 64 columns)
  if (!fp8_row_map(&a.x, xq, p.T, p.K, xq_stride, 128) ||
      !encode_tmap_2d(&a.out, Elem<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.out, (uint64_t)p.N,
                      (uint64_t)p.T, (uint64_t)p.out_stride * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  a.nm = (p.T + 127) / 128;
  a.nn = (p.N + 255) / 256;
  // A group's rows (16 MB, or eight tiles where these are more: K > 16384) stay in L2 while the weights stream past them; more
  // than 64 tiles leave too few weight tiles at work at a time.  8192 x 1536 -> 24576: 238 us in one group of 64, as here,
  // 253 in groups of 18; 16384 x 7168 -> 2112: 222 in groups of 18, as here, 199 of 24, 247 of 64, 265 in one of 128; 16384 x
  // 512 -> 32768: 280-291 in groups of 64, as here, 290-299 of 24, 311-314 in one of 128.
  const long long fit = (1ll << 24) / (128ll * p.K);
  a.group = fit < 8 ? 8 : fit > 64 ? 64 : (int)fit;
  const long long tiles = (long long)a.nm * a.nn;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(tiles < num_sms ? (int)tiles : num_sms);
  c.blockDim = dim3(kWdThreads);
  c.dynamicSmemBytes = kWdSmem;
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = p.dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, fp8_wide_kernel<T>, a);
}

}  // namespace

cudaError_t fp8_wide_prepare() {
  const void* k[2] = {(const void*)fp8_wide_kernel<__half>, (const void*)fp8_wide_kernel<__nv_bfloat16>};
  for (const void* f : k) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, f);
    if (e != cudaSuccess) return e;
    // (with fewer registers at launch the epilogue warps would wait for theirs for ever)
    if (at.numRegs * kWdThreads < 128 * kWdRoleRegs + 512 * kWdEpiRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kWdSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t fp8_wide_launch(bool bf16, const Fp8LinearParams& p, const CUtensorMap& w, const void* xq, int xq_stride, int num_sms,
                            cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, w, xq, xq_stride, num_sms, stream) : launch<__half>(p, w, xq, xq_stride, num_sms, stream);
}

}  // namespace mla
