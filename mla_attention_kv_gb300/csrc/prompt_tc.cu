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
// A CTA takes 128 query rows of a head and loads their keys and values by
// itself, 80 KB a tile, mostly from L2 (hit rate 83 %): neighbours take
// neighbouring blocks of a head, so a tile is wanted by several at about the
// same time.  Copies shared by a pair of CTAs were worth 1 to 4 % (8192 tokens,
// 128 heads: 1.86 to 1.89 ms) and would bind the operator to memory of the
// GPU that it runs on.
//
// Tensor memory: scores S0, S1 (128 columns each, by the parity of the key
// tile; the rounded weights overwrite the first 64 columns of theirs and are
// the A operand of the second product), output (128), queries (96).  With both
// A operands in tensor memory an MMA of 128 x 128 x 16 takes 64 cycles, so a
// tile of 128 keys needs 1280, and all of shared memory holds keys (three
// stages of 48 KB: three blocks of 64 columns, 128 bytes a row, 128-byte
// swizzle) and values (two stages of 32 KB).  One barrier per stage: a wait on
// an mbarrier takes a thread about 100 cycles even when the phase is complete,
// so finer slots cost more than they hide.
//
// What bounds it (one prompt of 8192, 128 heads, causal, bf16: 1.91 to 1.95
// ms, 1.42 PFLOP/s): 0.97 us per tile (about 1900 cycles), 1.8 us more per item
// and 17 us per call (fitted to non-causal prompts of 512 to 4096 tokens), the tensor
// pipe busy 60 % of the time.  A tile's way is scores, softmax, weights
// announced, output, with two tiles in flight.  Measured and slower: pairs of
// CTAs on the 2-SM MMA (half the shared-memory traffic, but every announcement
// crosses the CTAs) 1.99 ms; and, with pairs that shared their copies, four
// softmax warps per 32 rows 2.10 ms; tiles of 64 keys, four in flight, 2.10 ms.
//
// MMA order: scores of tile i + 1, then output of tile i, so the softmax of
// a tile runs under the scores of the next and the output of the previous.
// The CTAs are persistent: copies and scores of the next item begin while
// the last one's result is stored.
//
// The output is rescaled only when a row's maximum has grown by more than 2^8
// since the last time: rare after the first tiles.  A weight is then at most
// 2^8 (fp16 holds up to 65504), and the sums of weights and products are fp32.
//
// Warps: 0-7 queries, softmax, results (a row belongs to two threads, 64 keys
// of a tile each: warps q and q + 4), 8 TMA, 9 MMA.  Value rows past the
// sequence's end (tokens of no or another sequence, which may hold anything)
// are zeroed in shared memory by the softmax warps before the MMA reads them;
// scores of such keys are masked.  Keys that only later tokens of the sequence
// see are multiplied by a weight of 0, so their values have to be finite.
#include <string.h>

#include "attn.h"
#include "attn_tc.cuh"
#include "prompt_plan.cuh"
#include "tma.h"

namespace mla {
namespace {

constexpr int kPtThreads = kPromptPlanThreads;
constexpr int kPtTile = 128;   // query rows per CTA, keys per tile
constexpr int kKStages = 3, kVStages = 2;
constexpr uint32_t kBlock = 16384;  // 128 keys x 64 columns
constexpr uint32_t kKBytes = 3 * kBlock, kVBytes = 2 * kBlock;
constexpr uint32_t kPtV = kKStages * kKBytes;
constexpr uint32_t kPtBar = kPtV + kVStages * kVBytes;
constexpr uint32_t kPtSmem = kPtBar + 5120 + 1024;  // + alignment slack
static_assert(kPtSmem <= 232448, "shared memory of one CTA");
constexpr uint32_t kTmO = 256, kTmQ = 384;  // tensor memory columns; S0 at 0, S1 at 128
constexpr float kRescale = 8.0f;  // log2 of the growth of the maximum that rescales the output

struct PtShared {
  uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages];
  uint64_t sfull[2], pfull[2];
  uint64_t qready, ofree, pvdone, olast, done, pair[4];
  float row[2][2][128];  // exchange between the two threads of a row: [parity of the meeting][half][row]
  PromptPlan plan;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PtShared) <= 5120, "barrier block");

struct PtArgs {
  CUtensorMap kn, kp, v;
  PromptParams p;
};

template <typename T>
__global__ void __launch_bounds__(kPtThreads, 1)
    prompt_tc_kernel(const __grid_constant__ PtArgs a) {
  using E = Elem<T>;
  const PromptParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  PtShared* sh = reinterpret_cast<PtShared*>(smem + kPtBar);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };

  // the items of this CTA, with n key tiles each (n > 0: an item has a row, and a row sees a key)
  const int blocks = prompt_plan(p, &sh->plan, kPtTile, blockIdx.x == 0);
  const int cta = blockIdx.x;
  const long long items = (long long)blocks * p.heads;
  if (cta >= items) return;
  struct Item {
    PromptPlace pl;
    int n;
  };
  auto item_at = [&](long long x) {
    Item it;
    it.pl = prompt_place(p, &sh->plan, x, blocks, kPtTile);
    const int end = p.causal ? min(it.pl.len, it.pl.row0 + kPtTile) : it.pl.len;
    it.n = (end + kPtTile - 1) / kPtTile;
    return it;
  };

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(bar(&sh->kfull[i]), 1);
      mbar_init(bar(&sh->kempty[i]), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(bar(&sh->vfull[i]), 1);
      mbar_init(bar(&sh->vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh->sfull[i]), 1);
      mbar_init(bar(&sh->pfull[i]), 8);
    }
    mbar_init(bar(&sh->qready), 8);
    mbar_init(bar(&sh->ofree), 8);
    for (int i = 0; i < 4; ++i) mbar_init(bar(&sh->pair[i]), 2);
    mbar_init(bar(&sh->pvdone), 1);
    mbar_init(bar(&sh->olast), 1);
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(smem_u32(&sh->tmem), 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  if (warp == 8) {
    // ============================================================ TMA
    if (tc::elect_one()) {
      int nk = 0, nv = 0;  // stages filled
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const long long x = prompt_item(cta, p.ctas, k);
        if (x >= items) break;
        const Item it = item_at(x);
        const int hk = it.pl.head / (p.heads / p.kv_heads), t0 = it.pl.begin;
        auto keys = [&](int i) {
          const uint32_t s = nk % kKStages, b = bar(&sh->kfull[s]), d = sbase + s * kKBytes;
          ok = ok && at_wait(bar(&sh->kempty[s]), ((nk / kKStages) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) return;
          const int tok = t0 + i * kPtTile;
          mbar_arrive_expect_tx(b, kKBytes);
          tma_load_4d(d, &a.kn, 0, tok, hk, it.pl.batch, b);
          tma_load_4d(d + kBlock, &a.kn, 64, tok, hk, it.pl.batch, b);
          tma_load_4d(d + 2 * kBlock, &a.kp, 0, tok, 0, it.pl.batch, b);
          ++nk;
        };
        auto values = [&](int i) {
          const uint32_t s = nv % kVStages, b = bar(&sh->vfull[s]), d = sbase + kPtV + s * kVBytes;
          ok = ok && at_wait(bar(&sh->vempty[s]), ((nv / kVStages) & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) return;
          const int tok = t0 + i * kPtTile;
          mbar_arrive_expect_tx(b, kVBytes);
          tma_load_4d(d, &a.v, 0, tok, hk, it.pl.batch, b);
          tma_load_4d(d + kBlock, &a.v, 64, tok, hk, it.pl.batch, b);
          ++nv;
        };
        keys(0);
        for (int i = 0; i < it.n && ok; ++i) {
          if (i + 1 < it.n) keys(i + 1);
          values(i);
        }
      }
      // every copy has landed, and every release of a stage has arrived, before the CTA may exit
      const uint64_t t0 = globaltimer_ns();
      auto drain = [&](uint64_t* b, int use, int stages) {
        const uint64_t spent = globaltimer_ns() - t0, limit = drain_budget(p.budget_ns);
        mbar_wait_bounded(bar(b + use % stages), (use / stages) & 1, spent < limit ? limit - spent : 0);
      };
      for (int v = max(0, nk - kKStages); v < nk; ++v) {
        drain(sh->kfull, v, kKStages);
        drain(sh->kempty, v, kKStages);
      }
      for (int v = max(0, nv - kVStages); v < nv; ++v) {
        drain(sh->vfull, v, kVStages);
        drain(sh->vempty, v, kVStages);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ============================================================ MMA (one thread)
    if (tc::elect_one()) {
      const uint32_t id_qk = tc::idesc_f16(E::kBf16, 128, 128, false, false);
      const uint32_t id_pv = tc::idesc_f16(E::kBf16, 128, 128, false, true);
      const uint64_t dk = tc::sdesc_sw128(sbase, 16, 1024);             // K-major: keys
      const uint64_t dv = tc::sdesc_sw128(sbase + kPtV, kBlock, 1024);  // MN-major: values
      bool ok = at_wait_poll(bar(&sh->qready), 0, abort, p.budget_ns, p.status);
      auto wait = [&](uint64_t* b, uint32_t par) {
        ok = ok && at_wait(bar(b), par, abort, p.budget_ns, p.status);
        return ok;
      };
      uint32_t ks = 0, kp = 0, vs = 0, vp = 0;  // stage and phase of the rings
      uint32_t g_qk = 0, g_pv = 0, mine = 0;    // tiles done, items
      auto qk = [&]() {  // S = Q K^T
        if (!wait(&sh->kfull[ks], kp)) return;
        const uint64_t bd = dk + ks * (kKBytes >> 4);
        const uint32_t d = tmem + (g_qk & 1) * 128;
#pragma unroll 1
        for (int c = 0; c < 3; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f16_ts(d, tmem + kTmQ + c * 32 + k * 8, bd + c * (kBlock >> 4) + 2 * k, id_qk, c > 0 || k > 0);
        tc::commit(bar(&sh->sfull[g_qk & 1]));
        ++g_qk;
        tc::commit(bar(&sh->kempty[ks]));
        if (++ks == kKStages) {
          ks = 0;
          kp ^= 1;
        }
      };
      auto pv = [&](bool first, bool last) {  // O (+)= P V
        if (!wait(&sh->vfull[vs], vp)) return;
        // (the item before this one has been read from O)
        if (first && mine > 0 && !wait(&sh->ofree, (mine - 1) & 1)) return;
        if (!wait(&sh->pfull[g_pv & 1], (g_pv >> 1) & 1)) return;
        tc::fence_after_sync();
        const uint64_t bd = dv + vs * (kVBytes >> 4);
        const uint32_t pa = tmem + (g_pv & 1) * 128;
#pragma unroll 2
        for (int k = 0; k < 8; ++k) tc::mma_f16_ts(tmem + kTmO, pa + k * 8, bd + k * 128, id_pv, !first || k > 0);
        tc::commit(bar(&sh->pvdone));
        if (last) tc::commit(bar(&sh->olast));
        ++g_pv;
        tc::commit(bar(&sh->vempty[vs]));
        if (++vs == kVStages) {
          vs = 0;
          vp ^= 1;
        }
      };
      for (int k = 0; ok; ++k) {
        const long long x = prompt_item(cta, p.ctas, k);
        if (x >= items) break;
        const Item it = item_at(x);
        if (!wait(&sh->qready, mine & 1)) break;
        tc::fence_after_sync();
        qk();
        for (int i = 0; i < it.n && ok; ++i) {
          if (i + 1 < it.n) qk();
          if (ok) pv(i == 0, i == it.n - 1);
        }
        ++mine;
      }
      // every MMA issued so far has completed before TMEM is released
      tc::commit(bar(&sh->done));
      mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));
    }
    __syncwarp();
  } else {
    // ============================================================ queries, softmax, results
    const int q = warp & 3, hf = warp >> 2;
    const int r = q * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    const float scale = p.scale_log2;
    bool ok = true;
    // A row's 24 16-byte units of q_nope and q_pe: 12 to each of its two threads.
    auto q_unit = [&](const Item& it, int i) {
      const int u = hf * 12 + i;
      const bool pe = u >= 16;
      const PromptTensor& t = pe ? p.q_pe : p.q_nope;
      const int qi = it.pl.row0 + r;
      const int tok = it.pl.begin + (qi < it.pl.len ? qi : 0);
      return reinterpret_cast<const uint4*>(static_cast<const T*>(t.ptr) + (size_t)it.pl.batch * t.sb + (size_t)it.pl.head * t.sh + (size_t)tok * t.st) + (pe ? u - 16 : u);
    };
    auto load_q = [&](const Item& it) {
      const bool live = it.pl.row0 + r < it.pl.len;
      uint4 v[12];
#pragma unroll
      for (int i = 0; i < 12; ++i) v[i] = live ? *q_unit(it, i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 3; ++i) tc::st16(tl + kTmQ + hf * 48 + i * 16, reinterpret_cast<const uint32_t*>(v + 4 * i));
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh->qready));
    };
    uint32_t meets = 0;
    auto meet = [&]() {  // the two warps of these rows
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh->pair[q]));
      return at_wait_warp(bar(&sh->pair[q]), meets++ & 1, abort, p.budget_ns, p.status);
    };
    uint32_t g = 0, mine = 0;  // tiles, items done
    Item it = item_at(prompt_item(cta, p.ctas, 0));
    load_q(it);
    for (int round = 0; ok; ++round) {
      const long long xn = prompt_item(cta, p.ctas, round + 1);
      const bool more = xn < items;
      Item nx = it;
      if (more) {
        nx = item_at(xn);
        for (int i = 0; i < 12; i += 4)  // the next queries' lines into L2
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q_unit(nx, i)));
      }
      const int n = it.n;
      const int qi = it.pl.row0 + r;  // query's token in its sequence
      const bool live = qi < it.pl.len;
      float m = -INFINITY;  // maximum the weights are relative to (raw score units)
      float l = 0.f;        // sum over this thread's keys
      for (int i = 0; i < n; ++i, ++g) {
        const uint32_t ts = tl + (g & 1) * 128;
        if (!at_wait_warp(bar(&sh->sfull[g & 1]), (g >> 1) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
        tc::fence_after_sync();
        uint32_t s[64];
        tc::ld32(ts + hf * 64, s);
        tc::ld32(ts + hf * 64 + 32, s + 32);
        tc::wait_ld();
        // keys this row sees among this thread's 64
        const int limit = (p.causal ? min(qi + 1, it.pl.len) : it.pl.len) - i * kPtTile - hf * 64;
        if (__any_sync(~0u, limit < 64)) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (k >= limit) s[k] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(s[k]);
#pragma unroll
        for (int k = 4; k < 60; k += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], __uint_as_float(s[k + j]), __uint_as_float(s[k + j + 4]));
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], __uint_as_float(s[60 + j]));
        float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const uint32_t par = meets & 1;
        sh->row[par][hf][r] = tile_max;
        // both threads of a row have their scores in registers and their maxima in place
        if (!meet()) { ok = false; break; }
        tile_max = fmaxf(tile_max, sh->row[par][hf ^ 1][r]);
        if (__any_sync(~0u, (tile_max - m) * scale > kRescale)) {
          const float m_new = fmaxf(m, tile_max);
          const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * scale);
          if (i > 0) {
            if (!at_wait_warp(bar(&sh->pvdone), (g - 1) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
            tc::fence_after_sync();
            tmem_scale<64>(tl + kTmO + hf * 64, f);
            tc::wait_st();
          }
          l *= f;
          m = m_new;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t sc2 = f2_pack(scale, scale), ng2 = f2_pack(-mu * scale, -mu * scale);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
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
          tc::st16(ts + hf * 32 + c * 16, pk);
        }
        tc::wait_st();
        tc::fence_before_sync();
        const int valid = it.pl.len - i * kPtTile;
        if (valid < kPtTile) {
          // value rows past the sequence's end: whole 128-byte rows, so the swizzle does not matter
          const uint32_t vs = g % kVStages;
          if (!at_wait_warp(bar(&sh->vfull[vs]), (g / kVStages) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
          for (int x = tid; x < (kPtTile - valid) * 16; x += 256)
            *reinterpret_cast<uint4*>(smem + kPtV + vs * kVBytes + ((x >> 3) & 1) * kBlock + (valid + x / 16) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh->pfull[g & 1]));
        float a0, a1, b0, b1;
        f2_unpack(sum[0], a0, a1);
        f2_unpack(sum[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
      }
      if (!ok) break;
      // the next item's queries go in while the last output MMA runs (all score MMAs of this one are done)
      if (more) load_q(nx);
      {
        const uint32_t par = meets & 1;
        sh->row[par][hf][r] = l;
        // (a barrier of its own: a parity says which of two neighbouring phases is done, and this warp has not followed
        // those of pvdone)
        ok = meet() && at_wait_warp(bar(&sh->olast), mine++ & 1, abort, p.budget_ns, p.status);
        if (!ok) break;
        tc::fence_after_sync();
        l = sh->row[par][0][r] + sh->row[par][1][r];
        const float iv = l == 0.f ? 0.f : 1.f / l;
        const int tok = it.pl.begin + (live ? qi : 0);
        T* out = static_cast<T*>(const_cast<void*>(p.out.ptr)) + (size_t)it.pl.batch * p.out.sb + (size_t)it.pl.head * p.out.sh + (size_t)tok * p.out.st + hf * 64;
        uint32_t o[64];
        tc::ld32(tl + kTmO + hf * 64, o);
        tc::ld32(tl + kTmO + hf * 64 + 32, o + 32);
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&sh->ofree));
        if (live) {
#pragma unroll
          for (int k = 0; k < 64; k += 8) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = E::pack(__uint_as_float(o[k + 2 * j]) * iv, __uint_as_float(o[k + 2 * j + 1]) * iv);
            *reinterpret_cast<uint4*>(out + k) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (hf == 0 && p.lse)
            p.lse[((size_t)it.pl.batch * p.heads + it.pl.head) * p.s + tok] = l == 0.f ? -INFINITY : (m * scale + log2f(l)) * kLn2;
        }
      }
      if (!more) break;
      it = nx;
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
  const PromptTensor* src[3] = {&p.k_nope, &p.k_pe, &p.value};
  for (int i = 0; i < 3; ++i) key.t[i] = *src[i];
  key.b = p.b; key.s = p.s; key.kv_heads = p.kv_heads;
  if (!m->valid || memcmp(&key, &m->key, sizeof(key)) != 0) {
    m->valid = false;
    const int width[3] = {kNope, kRope, kV};
    const int heads[3] = {p.kv_heads, 1, p.kv_heads};
    const CUtensorMapDataType dt = Elem<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    for (int i = 0; i < 3; ++i) {
      const PromptTensor& t = *src[i];
      if (!encode_tmap_4d_rows(&m->map[i], dt, t.ptr, width[i], p.s, heads[i], p.b, t.st, heads[i] > 1 ? t.sh : width[i], t.sb, kPtTile))
        return cudaErrorInvalidValue;
    }
    m->key = key;
    m->valid = true;
  }
  PtArgs a;
  a.kn = m->map[0]; a.kp = m->map[1]; a.v = m->map[2];
  a.p = p;
  const long long items = (long long)prompt_blocks(p, kPtTile) * p.heads;
  if (items < a.p.ctas) a.p.ctas = (int)items;
  prompt_tc_kernel<T><<<a.p.ctas, kPtThreads, kPtSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prompt_tc_prepare(bool bf16) {
  return bf16 ? cudaFuncSetAttribute(prompt_tc_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPtSmem)
              : cudaFuncSetAttribute(prompt_tc_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPtSmem);
}

cudaError_t prompt_tc_launch(bool bf16, const PromptParams& p, PromptMaps* maps, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, maps, stream) : launch<__half>(p, maps, stream);
}

}  // namespace mla
