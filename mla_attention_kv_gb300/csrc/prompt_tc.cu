// prompt_tc.cu -- attention over whole prompts in the up-projected form, on
// tcgen05 / TMEM / TMA.
//
// Per query row (token i, head h; q = [q_nope 128 | q_pe 64]) and key token
// j of the same sequence (k = [k_nope 128 of head h's group | k_pe 64 shared
// by all heads], value 128): out = sum_j softmax(scale * q . k_j) value_j
// over j <= i (causal) or all j.  One pass over the keys with a running
// maximum and sum per row in fp32; the weights are rounded to the I/O dtype
// for their product with the values (the operand type of the MMA), the sum
// takes them before that.
//
// One CTA per 256 query rows of a head, as two tiles of 128 that share every
// key tile (128 keys) and take turns on the tensor core: while one tile's
// scores are in the softmax warps the other tile's MMAs run.  Per pair of
// 128 x 128 tiles the MMA needs 2 * (768 + 512) cycles (QK: 12 steps of
// K = 16, PV: 8), the softmax one exponential per score.
//
// Tensor memory (512 columns): S0, S1 (128 each, fp32 scores; the rounded
// weights overwrite the first 64 columns of theirs and are the A operand of
// the PV MMA), O0, O1 (128 each).  Shared memory: the queries (96 KB) and a
// ring of eight 16 KB slots; a key tile is three slots (64 columns each, 128
// bytes a row, 128-byte swizzle), its values two.
//
// The output is rescaled only when a row's maximum has grown by more than 2^8
// since the last time (weights are then at most 2^8: the sums stay exact to
// fp32 and 2^8 * 128 keys is far inside fp16's range): rare after the first
// tiles.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1 (a thread owns a row), 8 TMA,
// 9 MMA.  Value rows past the sequence's end (tokens of no or another
// sequence, which may hold anything) are zeroed in shared memory by warp 9
// before the MMA reads them; scores of such keys are masked.
#include <string.h>

#include "attn.h"
#include "attn_tc.cuh"
#include "prompt_plan.cuh"
#include "tma.h"

namespace mla {
namespace {

constexpr int kPtThreads = 320;
constexpr int kPtRows = 256;   // query rows per CTA
constexpr int kPtTile = 128;   // query rows per MMA tile, keys per tile
constexpr int kPtSlots = 8;
constexpr uint32_t kPtSlotBytes = 16384;
constexpr uint32_t kPtQBytes = 3 * 16384;  // one tile's queries
constexpr uint32_t kPtRing = 2 * kPtQBytes;
constexpr uint32_t kPtBar = kPtRing + kPtSlots * kPtSlotBytes;
constexpr uint32_t kPtSmem = kPtBar + 512 + 1024;  // + alignment slack
static_assert(kPtSmem <= 232448, "shared memory of one CTA");
constexpr float kRescale = 8.0f;  // log2 of the growth of the maximum that rescales the output

struct PtShared {
  uint64_t full[kPtSlots], empty[kPtSlots];
  uint64_t qfull[2], sfull[2], pfull[2], ofull[2];
  uint64_t done;
  PromptPlanShared plan;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PtShared) <= 512, "barrier block");

struct PtArgs {
  CUtensorMap qn, qp, kn, kp, v;
  PromptParams p;
};

template <typename T>
__global__ void __launch_bounds__(kPtThreads, 1) prompt_tc_kernel(const __grid_constant__ PtArgs a) {
  using E = Elem<T>;
  const PromptParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  PtShared* sh = reinterpret_cast<PtShared*>(smem + kPtBar);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };

  PromptPlace pl;
  if (!prompt_place(p, &sh->plan, blockIdx.x, kPtRows, &pl, blockIdx.x == 0 && blockIdx.y == 0)) return;
  const int h = blockIdx.y, hk = h / (p.heads / p.kv_heads);
  // key tiles of the two query tiles (tile 1 may have no rows)
  const int rows = min(kPtRows, pl.len - pl.row0);
  auto tiles_of = [&](int w) {
    if (w * kPtTile >= rows) return 0;
    const int end = p.causal ? min(pl.len, pl.row0 + (w + 1) * kPtTile) : pl.len;
    return (end + kPtTile - 1) / kPtTile;
  };
  const int n0 = tiles_of(0), n1 = tiles_of(1), nt = max(n0, n1);

  if (tid == 0) {
    for (int i = 0; i < kPtSlots; ++i) {
      mbar_init(bar(&sh->full[i]), 1);
      mbar_init(bar(&sh->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh->qfull[i]), 1);
      mbar_init(bar(&sh->sfull[i]), 1);
      mbar_init(bar(&sh->pfull[i]), 4);
      mbar_init(bar(&sh->ofull[i]), 1);
    }
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(smem_u32(&sh->tmem), 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh->tmem;

  if (warp == 8) {
    // ============================================================ TMA
    if (lane == 0) {
      for (int w = 0; w < 2; ++w) {
        if ((w ? n1 : n0) == 0) continue;
        const uint32_t q = sbase + w * kPtQBytes, b = bar(&sh->qfull[w]);
        const int tok = pl.begin + pl.row0 + w * kPtTile;
        mbar_arrive_expect_tx(b, kPtQBytes);
        tma_load_4d(q, &a.qn, 0, tok, h, pl.batch, b);
        tma_load_4d(q + 16384, &a.qn, 64, tok, h, pl.batch, b);
        tma_load_4d(q + 32768, &a.qp, 0, tok, h, pl.batch, b);
      }
      uint32_t u = 0;
      bool ok = true;
      for (int i = 0; i < nt && ok; ++i) {
        const int tok = pl.begin + i * kPtTile;
        for (int c = 0; c < 5; ++c, ++u) {
          const uint32_t s = u % kPtSlots;
          if (!at_wait(bar(&sh->empty[s]), ((u / kPtSlots) & 1) ^ 1, abort, p.budget_ns, p.status)) { ok = false; break; }
          const uint32_t d = sbase + kPtRing + s * kPtSlotBytes, b = bar(&sh->full[s]);
          mbar_arrive_expect_tx(b, kPtSlotBytes);
          if (c < 2) tma_load_4d(d, &a.kn, c * 64, tok, hk, pl.batch, b);
          else if (c == 2) tma_load_4d(d, &a.kp, 0, tok, 0, pl.batch, b);
          else tma_load_4d(d, &a.v, (c - 3) * 64, tok, hk, pl.batch, b);
        }
      }
      // every issued copy has landed before the CTA may exit
      for (uint32_t v = u > kPtSlots ? u - kPtSlots : 0; v < u; ++v)
        mbar_wait_bounded(bar(&sh->full[v % kPtSlots]), (v / kPtSlots) & 1, drain_budget(p.budget_ns));
      for (int w = 0; w < 2; ++w)
        if ((w ? n1 : n0) > 0) mbar_wait_bounded(bar(&sh->qfull[w]), 0, drain_budget(p.budget_ns));
    }
  } else if (warp == 9) {
    // ============================================================ MMA (whole warp; an elected lane issues)
    const uint32_t id_qk = tc::idesc_f16(E::kBf16, 128, 128, false, false);
    const uint32_t id_pv = tc::idesc_f16(E::kBf16, 128, 128, false, true);
    const uint32_t id_pv64 = tc::idesc_f16(E::kBf16, 128, 64, false, true);
    const uint64_t dk0 = tc::sdesc_sw128(sbase, 16, 1024);            // K-major: queries, keys
    const uint64_t dv0 = tc::sdesc_sw128(sbase, kPtSlotBytes, 1024);  // MN-major: values
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t par) {
      ok = ok && at_wait_warp(bar(b), par, abort, p.budget_ns, p.status);
      return ok;
    };
    auto slot_full = [&](uint32_t u) { return wait(&sh->full[u % kPtSlots], (u / kPtSlots) & 1); };
    auto qk = [&](int w, int i) {  // S_w = Q_w K_i^T
      for (int c = 0; c < 3; ++c) {
        const uint32_t u = 5 * i + c;
        if (!slot_full(u)) return;
        if (tc::elect_one()) {
          const uint64_t ad = dk0 + ((w * kPtQBytes + c * 16384) >> 4);
          const uint64_t bd = dk0 + ((kPtRing + (u % kPtSlots) * kPtSlotBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::mma_f16(tmem + w * 128, ad + 2 * k, bd + 2 * k, id_qk, c > 0 || k > 0);
        }
      }
      if (tc::elect_one()) tc::commit(bar(&sh->sfull[w]));
      __syncwarp();
    };
    auto release = [&](uint32_t u, int n) {
      if (tc::elect_one())
        for (int c = 0; c < n; ++c) tc::commit(bar(&sh->empty[(u + c) % kPtSlots]));
      __syncwarp();
    };
    bool zeroed = false;
    auto pv = [&](int w, int i, bool last) {  // O_w += P_w V_i
      const uint32_t u = 5 * i + 3;
      if (!slot_full(u) || !slot_full(u + 1)) return;
      const int valid = pl.len - i * kPtTile;
      if (valid < kPtTile && !zeroed) {
        // rows past the sequence's end: whole 128-byte rows, so the swizzle does not matter
        for (int x = lane; x < (kPtTile - valid) * 16; x += 32) {
          const int r = valid + x / 16, c = x % 16;
          const uint32_t sl = (u + (c >> 3)) % kPtSlots;
          *reinterpret_cast<uint4*>(smem + kPtRing + sl * kPtSlotBytes + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        zeroed = true;
      }
      if (!wait(&sh->pfull[w], i & 1)) return;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint32_t s0 = u % kPtSlots, s1 = (u + 1) % kPtSlots;
        const uint64_t b0 = dv0 + ((kPtRing + s0 * kPtSlotBytes) >> 4), b1 = dv0 + ((kPtRing + s1 * kPtSlotBytes) >> 4);
        const uint32_t o = tmem + 256 + w * 128, pa = tmem + w * 128;
        if (s1 == s0 + 1) {
#pragma unroll
          for (int k = 0; k < 8; ++k) tc::mma_f16_ts(o, pa + k * 8, b0 + k * 128, id_pv, i > 0 || k > 0);
        } else {  // the pair wraps around the ring
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            tc::mma_f16_ts(o, pa + k * 8, b0 + k * 128, id_pv64, i > 0 || k > 0);
            tc::mma_f16_ts(o + 64, pa + k * 8, b1 + k * 128, id_pv64, i > 0 || k > 0);
          }
        }
        if (last) tc::commit(bar(&sh->ofull[w]));
      }
      __syncwarp();
    };
    if (n0 > 0 && wait(&sh->qfull[0], 0)) qk(0, 0);
    if (n1 > 0 && ok && wait(&sh->qfull[1], 0)) qk(1, 0);
    if (ok) release(0, 3);
    for (int i = 0; i < nt && ok; ++i) {
      if (i < n0) pv(0, i, i == n0 - 1);
      if (ok && i + 1 < n0) qk(0, i + 1);
      if (ok && i < n1) pv(1, i, i == n1 - 1);
      if (!ok) break;
      release(5 * i + 3, 2);
      if (i + 1 < n1) qk(1, i + 1);
      if (ok && i + 1 < nt) release(5 * (i + 1), 3);
    }
    // every MMA issued so far has completed before TMEM is released
    if (tc::elect_one()) {
      tc::commit(bar(&sh->done));
      mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));
    }
    __syncwarp();
  } else {
    // ============================================================ softmax
    const int w = warp >> 2;
    const int n = w ? n1 : n0;
    const int r = (warp & 3) * 32 + lane;
    const int qi = pl.row0 + w * kPtTile + r;  // query's token in its sequence
    const uint32_t ts = tmem + w * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = ts - w * 128 + 256 + w * 128;
    float m = -INFINITY;  // maximum the weights are relative to (raw score units)
    float l = 0.f;
    const float scale = p.scale_log2;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      if (!at_wait_warp(bar(&sh->sfull[w]), i & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
      tc::fence_after_sync();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) tc::ld32(ts + c, s + c);
      tc::wait_ld();
      // keys this row sees in this tile
      const int limit = (p.causal ? min(qi + 1, pl.len) : pl.len) - i * kPtTile;
      if (__any_sync(~0u, limit < kPtTile)) {
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k >= limit) s[k] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
      for (int k = 4; k < 128; k += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], __uint_as_float(s[k + j]));
      const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (__any_sync(~0u, (tile_max - m) * scale > kRescale)) {
        // (the MMA that filled S was issued after the last one that wrote O: O is at rest)
        const float m_new = fmaxf(m, tile_max);
        const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * scale);
        if (i > 0) {
          tmem_scale<128>(to, f);
          tc::wait_st();
        }
        l *= f;
        m = m_new;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      const uint64_t sc2 = f2_pack(scale, scale), ng2 = f2_pack(-mu * scale, -mu * scale);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = c * 32 + 2 * k;
          const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), sc2, ng2);
          float x0, x1;
          f2_unpack(x, x0, x1);
          x0 = ex2(x0);
          x1 = ex2(x1);
          sum[k & 1] = f2_add(sum[k & 1], f2_pack(x0, x1));
          pk[k] = E::pack(x0, x1);
        }
        tc::st16(ts + c * 16, pk);
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh->pfull[w]));
      float a0, a1, b0, b1;
      f2_unpack(sum[0], a0, a1);
      f2_unpack(sum[1], b0, b1);
      l += (a0 + a1) + (b0 + b1);
    }
    if (ok && n > 0 && at_wait_warp(bar(&sh->ofull[w]), 0, abort, p.budget_ns, p.status)) {
      tc::fence_after_sync();
      const bool live = w * kPtTile + r < rows;
      const float iv = l == 0.f ? 0.f : 1.f / l;
      const int tok = pl.begin + qi;
      T* out = static_cast<T*>(const_cast<void*>(p.out.ptr)) + (size_t)pl.batch * p.out.sb + (size_t)h * p.out.sh + (size_t)(live ? tok : 0) * p.out.st;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        tc::ld32(to + c, o);
        tc::wait_ld();
        if (live) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              q[j] = E::pack(__uint_as_float(o[k + 2 * j]) * iv, __uint_as_float(o[k + 2 * j + 1]) * iv);
            *reinterpret_cast<uint4*>(out + c + k) = make_uint4(q[0], q[1], q[2], q[3]);
          }
        }
      }
      if (live && p.lse)
        p.lse[((size_t)pl.batch * p.heads + h) * p.s + tok] = l == 0.f ? -INFINITY : (m * scale + log2f(l)) * kLn2;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

template <typename T>
cudaError_t launch(const PromptParams& p, PromptMaps* m, cudaStream_t stream) {
  PromptMaps::Key key;
  memset(&key, 0, sizeof(key));
  const PromptTensor* src[5] = {&p.q_nope, &p.q_pe, &p.k_nope, &p.k_pe, &p.value};
  for (int i = 0; i < 5; ++i) key.t[i] = *src[i];
  key.b = p.b; key.s = p.s; key.heads = p.heads; key.kv_heads = p.kv_heads;
  if (!m->valid || memcmp(&key, &m->key, sizeof(key)) != 0) {
    m->valid = false;
    const int width[5] = {kNope, kRope, kNope, kRope, kV};
    const int heads[5] = {p.heads, p.heads, p.kv_heads, 1, p.kv_heads};
    const CUtensorMapDataType dt = Elem<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    for (int i = 0; i < 5; ++i) {
      const PromptTensor& t = *src[i];
      if (!encode_tmap_4d_rows(&m->map[i], dt, t.ptr, width[i], p.s, heads[i], p.b, t.st, heads[i] > 1 ? t.sh : width[i], t.sb, kPtTile))
        return cudaErrorInvalidValue;
    }
    m->key = key;
    m->valid = true;
  }
  PtArgs a;
  a.qn = m->map[0]; a.qp = m->map[1]; a.kn = m->map[2]; a.kp = m->map[3]; a.v = m->map[4];
  a.p = p;
  cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPtSmem);
  if (e != cudaSuccess) return e;
  prompt_tc_kernel<T><<<dim3(prompt_blocks(p, kPtRows), p.heads), kPtThreads, kPtSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_tc_launch(bool bf16, const PromptParams& p, PromptMaps* maps, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, maps, stream) : launch<__half>(p, maps, stream);
}

}  // namespace mla
