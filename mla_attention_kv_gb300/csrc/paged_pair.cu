// paged_pair.cu -- attention of new tokens over the paged latent cache, for
// items of 128 query rows, on the 2-SM MMA (tcgen05.mma.cta_group::2,
// M = 128) / TMEM / TMA.
//
// The mathematics is that of paged_mma.cu: per query row (a token and a
// head; q = [q_latent | q_pe], 576 wide) softmax(scale * q . key) over the
// cached rows, times the rows' first 512 columns, in one pass with a running
// maximum and sum; the weights are rounded to the I/O dtype as the A operand
// of the product with the latents.
//
// The two CTAs of a cluster take 64 rows of an item each.  With M = 128 over
// the pair a CTA's tensor memory holds its 64 rows of an N-column result in
// 128 lanes x N / 2 columns (lanes 64-127: the upper half of the columns), so
// the whole 64 x 512 fp32 output takes 256 columns, scores of a tile of 128
// keys 64 (two buffers), and nothing is computed twice.  As the B operand
// each CTA holds its half of the keys for the scores (64 keys x 576 columns)
// and its half of the columns of all keys for the output (128 keys x 256).
// (One 128-row M per CTA would fill tensor memory with the output alone; two
// CTAs with half of the output and all of the scores each: 325 us below.)
//
// Shared memory: queries 72 KB, weights 16 KB, keys 72 KB (three slots of
// three 64-column blocks), values 64 KB (four slots of 32 keys); one tile of
// each, refilled slot by slot behind the MMAs, all with the 128-byte swizzle.
// MMA order: scores of tile t + 1, then output of tile t, so the softmax of a
// tile runs under the output of the one before.
//
// What bounds it: a tile's 36 score steps take 32 cycles each and its 16
// output MMAs 64, 2180 together (measured alone), but they read 240 KB of
// shared memory and 152 KB are written beside them, 3060 cycles at 128 bytes
// each; the kernel takes 3100 where the cache is in L2 and 3700 from HBM.
// Both key and value copies by TMA reached 30 bytes per cycle and SM (4500
// cycles a tile), so the values come by cp.async, on the load/store path.
// Requests into L2 ahead of the copies changed nothing.  Decode of 64
// sequences of up to 32768 keys, 128 heads, bf16 (1.15 GB of cache): 250 us,
// 4.6 TB/s; chunks of up to 512 tokens over 8192 keys: 1.01 ms, 1.44 PFLOP/s.
//
// Rescaling the output only when a maximum grew by more than 2^8: as in
// prompt_tc.cu.
//
// Warps: 0-3 queries, softmax, results (a row belongs to two threads, 64 keys
// of a tile each: warps w and w + 2), 4 key copies by TMA (or 10 and 11 by
// cp.async), 5 MMA (the even CTA's, for both), 6-9 value copies, a slot each.
// What the MMAs wait for is counted on the even CTA's barriers.  Value rows
// past the keys are zeros; scores of such keys are masked.
#include <string.h>

#include "attn.h"
#include "attn_tc.cuh"
#include "paged_plan.cuh"
#include "tma.h"

namespace mla {
namespace {

// kBox: the page size is a multiple of kBoxRows and the keys come by TMA;
// else by cp.async (two more warps).  64 sequences of up to 16384 keys, 128
// heads, bf16, TMA / cp.async: page 64 141 / 199 us, 32 142 / 200 us; 16 and 8
// by cp.async 201 us (boxes of 16 and 8 rows, in a kernel that TMA bounded
// more: 1.27 and 1.9 times the time of 32).
template <bool kBox> constexpr int kPpThreads = kBox ? 320 : 384;
constexpr int kPpRows = kPagedPairRows;  // 128 per pair
constexpr int kPpKeys = 128;           // keys of a tile
constexpr int kBoxRows = 32;           // cache rows of a TMA copy
constexpr uint32_t kBlk = 8192;  // 64 rows x 64 columns
constexpr int kKSlots = 3, kVSlots = 4;
constexpr uint32_t kKSlot = 3 * kBlk, kVSlot = 2 * kBlk;
constexpr uint32_t kPpQ = 0, kPpP = kPpQ + 9 * kBlk, kPpK = kPpP + 2 * kBlk, kPpV = kPpK + kKSlots * kKSlot,
                   kPpBar = kPpV + kVSlots * kVSlot, kPpSmem = kPpBar + 2048 + 1024;  // + alignment slack
static_assert(kPpSmem <= 232448, "shared memory of one CTA");
static_assert(sizeof(PlanShared) <= kKSlots * kKSlot, "the plan is made in the key slots before any copy");
constexpr uint32_t kTmS = 256;  // tensor memory columns: output at 0, scores at 256 and 320
constexpr float kRescale = 8.0f;

struct PpShared {
  uint64_t kfull[kKSlots], kempty[kKSlots], vfull[kVSlots], vempty[kVSlots];
  uint64_t sfull[2], qready, pfull, pvdone, done, pair[2];
  float row[2][2][64];  // exchange between the two threads of a row: [parity of the meeting][half][row]
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(PpShared) <= 2048, "barrier block");

struct PpArgs {
  CUtensorMap lat, kpe;
  PagedParams p;
};

template <typename T, bool kBox>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPpThreads<kBox>, 1) paged_pair_kernel(const __grid_constant__ PpArgs a) {
  using E = Elem<T>;
  const PagedParams& p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  PpShared* sh = reinterpret_cast<PpShared*>(smem + kPpBar);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int H = p.heads;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };
  const int rank = blockIdx.x & 1, w = blockIdx.x >> 1;  // (clusters are pairs of neighbours along x)

  PlanShared* plan = reinterpret_cast<PlanShared*>(smem + kPpK);
  grid_dep_launch_dependents();  // (the joining kernel may take its place)
  const long long total = plan_total(p, plan, kPpRows, blockIdx.x == 0);
  const int W = total > 0 ? plan_workers(total, p.workers, kPpRows) : 0;
  if (tid == 0 && rank == 0) plan_open_join(p, w);  // (before any wait)
  if (w >= W) return;
  const long long x0 = plan_worker_begin(total, w, W), x1 = plan_worker_begin(total, w + 1, W);
  PlanCursor first;
  first.seek(p, plan, kPpRows, x0);

  if (tid == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(bar(&sh->kfull[i]), kBox ? 1 : 4);  // (the copying warps of both CTAs)
      mbar_init(bar(&sh->kempty[i]), 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(bar(&sh->vfull[i]), 2);  // the copying warps of both CTAs
      mbar_init(bar(&sh->vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&sh->sfull[i]), 1);
      mbar_init(bar(&sh->pair[i]), 2);
    }
    mbar_init(bar(&sh->qready), 8);  // the softmax warps of both CTAs
    mbar_init(bar(&sh->pfull), 8);
    mbar_init(bar(&sh->pvdone), 1);
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) tc::tmem_alloc2(smem_u32(&sh->tmem), 512);
  // (the plan has been read: its place becomes key slots)
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers are initialised before any copy, commit or arrival reaches them
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  // the tiles [t0, t1) of an item that fall to this worker
  auto span = [&](const PlanCursor& c, int* t0, int* t1) {
    const int keys = c.q.keys_of_item(c.j, kPpRows, H);
    const int tiles = (keys + kPpKeys - 1) / kPpKeys;
    *t0 = c.tile_at(x0 > c.lo ? x0 : c.lo, tiles, kPpRows);
    *t1 = c.tile_at(x1 < c.hi ? x1 : c.hi, tiles, kPpRows);
    return keys;
  };

  // the cache row of a key (-1: past the keys, or in a block that there is not)
  auto row_of = [&](const PlanCursor& c, int k, int keys) {
    if (k >= keys) return -1;
    const int pg = k / p.page;
    const int blk = p.table[(size_t)c.s * p.table_stride + pg];
    if (blk < 0 || blk >= p.nblocks) {
      atomicOr(p.status, kStatusBadSlot);
      return -1;
    }
    return blk * p.page + (k - pg * p.page);
  };

  if (kBox && warp == 4) {
    // ============================================================ keys, by TMA
    const int zero_row = p.nblocks * p.page;  // past the end of the map: reads as zeros
    uint32_t u = 0, fills = 0;                // tiles, slots filled
    bool ok = true;
    PlanCursor c = first;
    for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kPpRows)) {
      int t0, t1;
      const int keys = span(c, &t0, &t1);
      // lane l < 4 holds the cache row of the l-th 32 keys of a tile (-1: past the keys)
      auto rows_of = [&](int tile) {
        const int k = tile * kPpKeys + lane * kBoxRows;
        if (lane >= kPpKeys / kBoxRows || tile >= t1 || k >= keys) return -1;
        const int r = row_of(c, k, keys);
        return r < 0 ? zero_row : r;
      };
      int row = rows_of(t0);
      for (int t = t0; t < t1 && ok; ++t, ++u) {
        const int next = rows_of(t + 1);
        const uint32_t boxes = __popc(__ballot_sync(~0u, row >= 0));
        for (int g = 0; g < kKSlots; ++g) {
          ok = ok && at_wait_warp(bar(&sh->kempty[g]), (u & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(&sh->kfull[g]), boxes * kBoxRows * 128 * 3);
          __syncwarp();
          if (lane >> 1 == rank && row >= 0) {  // this CTA's half of the keys
            const uint32_t d = sbase + kPpK + g * kKSlot + (lane & 1) * (kBlk / 2), b = tc::mapa(bar(&sh->kfull[g]), 0);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const int blk = 3 * g + j;
              tma_load_2d_pair(d + j * kBlk, blk < 8 ? &a.lat : &a.kpe, blk < 8 ? blk * 64 : 0, row, b);
            }
          }
          ++fills;
        }
        row = next;
      }
    }
    // Every copy has landed, and every release of a slot has arrived, before the CTAs may exit.  After a wait that ran
    // out the two CTAs may have filled different numbers of slots: a fill that the other CTA has not matched is never
    // released, and its waits take the whole limit, in which it lands.
    __syncwarp();
    const uint64_t t0 = globaltimer_ns();
    auto drain = [&](uint64_t* b, uint32_t par) {
      const uint64_t spent = globaltimer_ns() - t0, limit = drain_budget(p.budget_ns);
      mbar_wait_bounded(bar(b), par, spent < limit ? limit - spent : 0);
    };
    for (int i = 0; i < kKSlots; ++i) {
      const uint32_t n = ring_uses(fills, kKSlots, i);
      if (n == 0) break;
      if (rank == 0) drain(&sh->kfull[i], (n - 1) & 1);
      drain(&sh->kempty[i], (n - 1) & 1);
    }
  } else if (!kBox && warp > 9) {
    // ============================================================ keys, by cp.async: 32 of this CTA's 64 to a warp
    const int part = rank * 2 + warp - 10;  // which 32 keys of a tile
    uint32_t u = 0, fills = 0;
    bool ok = true;
    PlanCursor c = first;
    for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kPpRows)) {
      int t0, t1;
      const int keys = span(c, &t0, &t1);
      int row = row_of(c, t0 * kPpKeys + part * 32 + lane, t0 < t1 ? keys : 0);
      for (int t = t0; t < t1 && ok; ++t, ++u) {
        for (int g = 0; g < kKSlots; ++g) {
          ok = at_wait_warp(bar(&sh->kempty[g]), (u & 1) ^ 1, abort, p.budget_ns, p.status);
          if (!ok) break;
          // lane = 16-byte unit of the slot's three blocks (the last of all is k_pe)
          const bool pe = g == kKSlots - 1 && lane >= 16;
          const T* src = pe ? static_cast<const T*>(p.kpe) + (lane & 7) * 8 : static_cast<const T*>(p.latent) + g * 192 + lane * 8;
          const size_t rs = pe ? p.kpe_rs : p.lat_rs;
          const uint32_t d = sbase + kPpK + g * kKSlot + (lane >> 3) * kBlk + (part & 1) * (kBlk / 2);
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            const int cr = __shfl_sync(~0u, row, r);
            if (lane < 24) cp_async16(d + r * 128 + (((lane & 7) ^ (r & 7)) * 16), src + (size_t)max(cr, 0) * rs, cr < 0 ? 0 : 16);
          }
          cp_async_commit();
          ++fills;
          if (g > 0) {  // the slot before is there
            cp_async_wait<1>();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::arrive_operands(tc::mapa(bar(&sh->kfull[g - 1]), 0));
          }
        }
        row = row_of(c, (t + 1) * kPpKeys + part * 32 + lane, t + 1 < t1 ? keys : 0);
        cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0) tc::arrive_operands(tc::mapa(bar(&sh->kfull[kKSlots - 1]), 0));
      }
    }
    for (int i = 0; i < kKSlots; ++i) {  // the last releases have arrived
      const uint32_t n = ring_uses(fills, kKSlots, i);
      if (n == 0 || !mbar_wait_bounded(bar(&sh->kempty[i]), (n - 1) & 1, drain_budget(p.budget_ns))) break;
    }
  } else if (warp > 5) {
    // ============================================================ values, by cp.async: a warp fills a slot
    const int slot = warp - 6;
    const uint32_t empty = bar(&sh->vempty[slot]), lead = tc::mapa(bar(&sh->vfull[slot]), 0);
    uint32_t u = 0;
    bool ok = true;
    PlanCursor c = first;
    for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kPpRows)) {
      int t0, t1;
      const int keys = span(c, &t0, &t1);
      int row = row_of(c, t0 * kPpKeys + slot * 32 + lane, t0 < t1 ? keys : 0);
      for (int t = t0; t < t1; ++t, ++u) {
        ok = at_wait_warp(empty, (u & 1) ^ 1, abort, p.budget_ns, p.status);
        if (!ok) break;
        // lane = 16-byte unit of this CTA's columns 128 rank .. + 127 of either half of the latents
        const T* src = static_cast<const T*>(p.latent) + (lane >> 4) * 256 + rank * 128 + (lane & 15) * 8;
        const uint32_t d = sbase + kPpV + slot * kVSlot + (lane >> 3) * (kBlk / 2);
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
          const int cr = __shfl_sync(~0u, row, r);
          cp_async16(d + r * 128 + (((lane & 7) ^ (r & 7)) * 16), src + (size_t)max(cr, 0) * p.lat_rs, cr < 0 ? 0 : 16);
        }
        cp_async_commit();
        row = row_of(c, (t + 1) * kPpKeys + slot * 32 + lane, t + 1 < t1 ? keys : 0);
        cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::arrive_operands(lead);
      }
    }
    cp_async_wait<0>();
    if (u > 0) mbar_wait_bounded(empty, (u - 1) & 1, drain_budget(p.budget_ns));  // the last release has arrived
  } else if (warp == 5) {
    // ============================================================ MMA (one thread of the even CTA)
    if (rank == 0 && tc::elect_one()) {
      const uint32_t id_qk = tc::idesc_f16(E::kBf16, 128, 128, false, false);
      const uint32_t id_pv = tc::idesc_f16(E::kBf16, 128, 256, false, true);
      const uint64_t dq = tc::sdesc_sw128(sbase + kPpQ, 16, 1024), dk = tc::sdesc_sw128(sbase + kPpK, 16, 1024);
      const uint64_t dp = tc::sdesc_sw128(sbase + kPpP, 16, 1024), dv = tc::sdesc_sw128(sbase + kPpV, kBlk / 2, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t par) {
        ok = ok && at_wait<true>(bar(b), par, abort, p.budget_ns, p.status);
        return ok;
      };
      uint32_t g_qk = 0, g_pv = 0, item = 0;
      auto qk = [&]() {  // scores of tile g_qk
        const uint32_t d = tmem + kTmS + (g_qk & 1) * 64;
#pragma unroll 1
        for (int g = 0; g < kKSlots; ++g) {
          if (!wait(&sh->kfull[g], g_qk & 1)) return;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 12; ++k) {
            const uint32_t o = (k >> 2) * (kBlk >> 4) + 2 * (k & 3);
            tc::mma2_f16(d, dq + g * (kKSlot >> 4) + o, dk + g * (kKSlot >> 4) + o, id_qk, g > 0 || k > 0);
          }
          tc::commit2_both(bar(&sh->kempty[g]));
        }
        tc::commit2_both(bar(&sh->sfull[g_qk & 1]));
        ++g_qk;
      };
      auto pv = [&](bool first_tile) {  // output of tile g_pv
        if (!wait(&sh->pfull, g_pv & 1)) return;
        tc::fence_after_sync();
#pragma unroll 1
        for (int s = 0; s < kVSlots; ++s) {
          if (!wait(&sh->vfull[s], g_pv & 1)) return;
          tc::fence_after_sync();
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tc::mma2_f16(tmem + j * 128, dp + (s >> 1) * (kBlk >> 4) + 4 * (s & 1) + 2 * k,
                           dv + s * (kVSlot >> 4) + k * 128 + j * (kBlk >> 4), id_pv, !first_tile || s > 0 || k > 0);
          tc::commit2_both(bar(&sh->vempty[s]));
        }
        tc::commit2_both(bar(&sh->pvdone));
        ++g_pv;
      };
      PlanCursor c = first;
      for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kPpRows)) {
        int t0, t1;
        span(c, &t0, &t1);
        if (t0 >= t1) continue;
        ok = item == 0 ? at_wait_poll<true>(bar(&sh->qready), 0, abort, p.budget_ns, p.status) : wait(&sh->qready, item & 1);
        if (!ok) break;
        ++item;
        tc::fence_after_sync();
        qk();
        for (int t = t0; t < t1 && ok; ++t) {
          if (t + 1 < t1) qk();
          if (ok) pv(t == t0);
        }
      }
      tc::commit2_both(bar(&sh->done));
    }
    __syncwarp();
  } else if (warp < 4) {
    // ============================================================ queries, softmax, results
    const int r = tid & 63, hf = tid >> 6;  // row of this CTA's 64, half of a tile's keys
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    const float scale = p.scale_log2;
    uint32_t g = 0, meets = 0;  // tiles done
    bool ok = true;
    auto announce = [&](uint64_t* b) {  // to the MMA thread
      __syncwarp();
      if (lane == 0) tc::arrive_operands(tc::mapa(bar(b), 0));
    };
    auto meet = [&]() {  // the two warps of these rows
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&sh->pair[warp & 1]));
      return at_wait_warp(bar(&sh->pair[warp & 1]), meets++ & 1, abort, p.budget_ns, p.status);
    };
    auto load_q = [&](const PlanCursor& c) {  // a warp takes 16 of the 64 rows, lane = 16-byte unit
      for (int i = 0; i < 16; ++i) {
        const int qr = warp * 16 + i, row = c.j * kPpRows + rank * 64 + qr;
        const bool live = row < c.q.n * H;
        const int tok = live ? row / H : 0, hd = live ? row - tok * H : 0;
        const T* ql = static_cast<const T*>(p.q_lat) + (size_t)(c.q.begin + tok) * p.ql_ts + (size_t)hd * p.ql_hs;
        const T* qp = static_cast<const T*>(p.q_pe) + (size_t)(c.q.begin + tok) * p.qp_ts + (size_t)hd * p.qp_hs;
        const uint32_t d = sbase + kPpQ + (lane >> 3) * kBlk + qr * 128 + (((lane & 7) ^ (qr & 7)) * 16);
        cp_async16(d, ql + lane * 8, live ? 16 : 0);
        cp_async16(d + 4 * kBlk, ql + 256 + lane * 8, live ? 16 : 0);
        if (lane < 8) cp_async16(d + 8 * kBlk, qp + lane * 8, live ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      tc::fence_proxy_async_smem();
      announce(&sh->qready);
    };
    PlanCursor c = first;
    {
      int t0, t1;
      span(c, &t0, &t1);
      if (t0 < t1) load_q(c);
    }
    for (bool more = true; more && c.lo < x1 && ok;) {
      int t0, t1;
      span(c, &t0, &t1);
      if (tid == 0 && rank == 0 && c.hi >= x1) plan_post_join(p, c, kPpRows, w, x0, x1, total, W);
      const int row = c.j * kPpRows + rank * 64 + r;
      const int rows = min(32, c.q.n * H - (row - lane));  // of this warp's 32
      const bool live = lane < rows;
      const int limit0 = (live ? c.q.keys_of_row(row, H) : 0) - hf * 64;
      const bool whole = c.lo >= x0 && c.hi <= x1;
      const size_t grow = (size_t)c.q.begin * H + row;
      const size_t slot = (size_t)w * 2 + (c.lo < x0 ? 0 : 1);
      float m = -INFINITY, l = 0.f;  // maximum of the row, sum over this thread's keys
      for (int t = t0; t < t1; ++t, ++g) {
        const uint32_t ts = tl + kTmS + (g & 1) * 64;
        if (!at_wait_warp(bar(&sh->sfull[g & 1]), (g >> 1) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
        tc::fence_after_sync();
        uint32_t s[64];
        tc::ld32(ts, s);
        tc::ld32(ts + 32, s + 32);
        tc::wait_ld();
        const int limit = limit0 - t * kPpKeys;
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
        if (!meet()) { ok = false; break; }
        tile_max = fmaxf(tile_max, sh->row[par][hf ^ 1][r]);
        float f = 1.f;
        const bool grow_max = __any_sync(~0u, (tile_max - m) * scale > kRescale);  // (both warps of the rows alike)
        if (grow_max) {
          const float m_new = fmaxf(m, tile_max);
          f = m == -INFINITY ? 0.f : ex2((m - m_new) * scale);
          l *= f;
          m = m_new;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t sc2 = f2_pack(scale, scale), ng2 = f2_pack(-mu * scale, -mu * scale);
        uint64_t sum[2] = {0, 0};
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), sc2, ng2);
          float y0, y1;
          f2_unpack(x, y0, y1);
          y0 = ex2(y0);
          y1 = ex2(y1);
          sum[k & 1] = f2_add(sum[k & 1], f2_pack(y0, y1));
          pk[k] = E::pack(y0, y1);
        }
        float a0, a1, b0, b1;
        f2_unpack(sum[0], a0, a1);
        f2_unpack(sum[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        // the previous tile's output MMA has read the weights and left the output at rest
        if (g > 0 && !at_wait_warp(bar(&sh->pvdone), (g - 1) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
        tc::fence_after_sync();
        if (grow_max && t > t0) {
          tmem_scale<256>(tl, f);
          tc::wait_st();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(smem + kPpP + hf * kBlk + r * 128 + ((i ^ (r & 7)) * 16)) =
              make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        announce(&sh->pfull);
      }
      if (!ok) break;
      // the next item's queries go in while the last output MMA runs (all score MMAs of this one are done)
      more = c.next(p, kPpRows);
      if (more && c.lo < x1) {
        int u0, u1;
        span(c, &u0, &u1);
        if (u0 < u1) load_q(c);
      }
      if (t0 < t1) {
        const uint32_t par = meets & 1;
        sh->row[par][hf][r] = l;
        ok = meet() && at_wait_warp(bar(&sh->pvdone), (g - 1) & 1, abort, p.budget_ns, p.status);
        if (!ok) break;
        tc::fence_after_sync();
        l = sh->row[par][0][r] + sh->row[par][1][r];
      }
      // this thread's columns: 128 hf .. 128 hf + 127 of either half of the output
      const float iv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      if (t0 < t1) {
        // 32 columns at a time through the weights' place, so that a warp stores whole rows' pieces
        unsigned char* st = smem + kPpP + warp * 4096;
        T* out = static_cast<T*>(p.out) + (grow - lane) * kRank + hf * 128;  // (of the warp's first row)
        float* po = p.part_o + (slot * kPpRows + rank * 64 + (warp & 1) * 32) * kRank + hf * 128;
#pragma unroll 1
        for (int cc = 0; cc < 256; cc += 32) {
          uint32_t o[32];
          tc::ld32(tl + cc, o);
          tc::wait_ld();
          const int col = (cc >> 7) * 256 + (cc & 127);
          __syncwarp();
          if (whole) {  // four units of 16 bytes a row
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t q[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                q[j] = E::pack(__uint_as_float(o[8 * k + 2 * j]) * iv, __uint_as_float(o[8 * k + 2 * j + 1]) * iv);
              *reinterpret_cast<uint4*>(st + lane * 64 + ((k ^ (lane >> 1 & 3)) * 16)) = make_uint4(q[0], q[1], q[2], q[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = i * 8 + (lane >> 2), k = lane & 3;
              if (rr < rows)
                *reinterpret_cast<uint4*>(out + (size_t)rr * kRank + col + k * 8) = *reinterpret_cast<const uint4*>(st + rr * 64 + ((k ^ (rr >> 1 & 3)) * 16));
            }
          } else {  // eight units a row
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(st + lane * 128 + ((k ^ (lane & 7)) * 16)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3), k = lane & 7;
              if (rr < rows)
                *reinterpret_cast<uint4*>(po + (size_t)rr * kRank + col + k * 4) = *reinterpret_cast<const uint4*>(st + rr * 128 + ((k ^ (rr & 7)) * 16));
            }
          }
        }
        tc::fence_before_sync();
      } else if (whole && live) {  // no key at all
        T* out = static_cast<T*>(p.out) + grow * kRank + hf * 128;
        for (int cc = 0; cc < 256; cc += 8)
          *reinterpret_cast<uint4*>(out + (cc >> 7) * 256 + (cc & 127)) = make_uint4(0, 0, 0, 0);
      }
      if (hf == 0 && live) {
        if (!whole) {
          float* ml = p.part_ml + (slot * kPpRows + rank * 64 + r) * 2;
          ml[0] = m * scale;
          ml[1] = l;
        } else if (p.lse) {
          p.lse[grow] = l == 0.f ? -INFINITY : (m * scale + log2f(l)) * kLn2;
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));  // every MMA issued has completed
  // neither CTA leaves, or releases the pair's tensor memory, while its peer may still copy into it, read it, or arrive
  // on its barriers
  tc::cluster_sync();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

template <typename T>
cudaError_t launch(const PagedParams& p, PagedMaps* m, cudaStream_t stream) {
  PagedMaps::Key key;
  memset(&key, 0, sizeof(key));
  key.lat = p.latent; key.kpe = p.kpe; key.lat_rs = p.lat_rs; key.kpe_rs = p.kpe_rs; key.rows = p.nblocks * p.page;
  const bool box = p.page % kBoxRows == 0;
  if (box && (!m->valid || memcmp(&key, &m->key, sizeof(key)) != 0)) {
    m->valid = false;
    const CUtensorMapDataType dt = Elem<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!encode_tmap_2d(&m->lat, dt, p.latent, kRank, key.rows, (uint64_t)p.lat_rs * 2, 64, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&m->kpe, dt, p.kpe, kRope, key.rows, (uint64_t)p.kpe_rs * 2, 64, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    m->key = key;
    m->valid = true;
  }
  PpArgs a;
  a.lat = m->lat; a.kpe = m->kpe; a.p = p;
  if (box)
    paged_pair_kernel<T, true><<<p.workers * 2, kPpThreads<true>, kPpSmem, stream>>>(a);
  else
    paged_pair_kernel<T, false><<<p.workers * 2, kPpThreads<false>, kPpSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t paged_pair_prepare(bool bf16) {
  const void* k[2] = {bf16 ? (const void*)paged_pair_kernel<__nv_bfloat16, true> : (const void*)paged_pair_kernel<__half, true>,
                      bf16 ? (const void*)paged_pair_kernel<__nv_bfloat16, false> : (const void*)paged_pair_kernel<__half, false>};
  for (const void* f : k) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kPpSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t paged_pair_launch(bool bf16, const PagedParams& p, PagedMaps* maps, cudaStream_t stream) {
  return bf16 ? launch<__nv_bfloat16>(p, maps, stream) : launch<__half>(p, maps, stream);
}

}  // namespace mla
