// paged_tc.cu -- attention of new tokens over the paged latent cache, for
// items of 128 query rows, on tcgen05 / TMEM / TMA.
//
// The mathematics is that of paged_mma.cu: per query row (a token and a
// head; q = [q_latent | q_pe], 576 wide) softmax(scale * q . key) over the
// cached rows, times the rows' first 512 columns, in one pass with a running
// maximum and sum; the weights are rounded to the I/O dtype as the A operand
// of the product with the latents.
//
// A 128 x 512 fp32 output alone would fill the 512 columns of tensor memory,
// so two CTAs share an item: both compute the scores, each accumulates half
// (256 columns) of the output, without any exchange.  (Half of the scores'
// columns each and an exchange of partial scores would save 35 % of the MMA
// cycles, but 32 KB per tile each way take 1700 cycles through distributed
// shared memory, measured at 19 bytes per cycle.)  Tensor memory: output
// [0, 256), scores of a 64-key tile [256, 320), the rounded weights
// [320, 352), and 320 of the queries' 576 columns [352, 512) as the A operand
// of their part of the scores; the other 256 stay in shared memory (64 KB),
// which leaves 160 KB for keys.
//
// What bounds it: a score step of 16 columns takes the tensor core 32 cycles
// with A in tensor memory and 48 with A in shared memory, an output step of 16
// keys 128, so a tile takes 20 * 32 + 16 * 48 + 4 * 128 = 1920; the kernel
// takes 2420.  Decode of 64 sequences of up to 32768 keys, 128 heads, bf16
// (1.15 GB of cache): 325 us, 3.5 TB/s.
//
// Keys: a tile is nine blocks of 64 keys x 64 columns (8 KB, 128-byte
// swizzle) by TMA, in boxes of 32 or 64 rows of a page.  Five blocks serve the scores alone and are released
// as soon as their MMAs are done (one stage); the four of this CTA's output
// half are the B operand of both products (three stages).  Tiles are
// requested into L2 four tiles ahead of their copies.
// MMA order: scores of tile i + 1, then output of tile i, so the softmax of
// a tile runs under the scores of the next.
//
// Rescaling the output only when a maximum grew by more than 2^8: as in
// prompt_tc.cu.
//
// Pages that such boxes do not fit: three warps copy row by row with cp.async
// into the same layout (the swizzle done by hand).
//
// Warps: 0-3 queries, softmax, results (a thread owns a row), 4 TMA (or 4, 6
// and 7 copies of rows), 5 MMA.
#include "attn.h"
#include "attn_tc.cuh"
#include "paged_plan.cuh"

namespace mla {
namespace {

constexpr int kUtThreads = 256;
constexpr int kCopyWarps = 3;
constexpr int kUtRows = kPagedTcRows;  // 128
constexpr uint32_t kBlk = 8192;        // 64 keys x 64 columns
constexpr int kNTiles = 1, kVTiles = 3;  // stages of the two rings
constexpr uint32_t kNBytes = 5 * kBlk, kVBytes = 4 * kBlk;
constexpr uint32_t kUtQ = 0;                              // 4 chunks of [128 x 64]
constexpr uint32_t kUtV = kUtQ + 4 * 16384;               // [kVTiles][4] blocks
constexpr uint32_t kUtN = kUtV + kVTiles * kVBytes;       // [kNTiles][5] blocks
constexpr uint32_t kUtBar = kUtN + kNTiles * kNBytes;
constexpr uint32_t kUtSmem = kUtBar + 512 + 1024;
static_assert(kUtSmem <= 232448, "shared memory of one CTA");
static_assert(sizeof(PlanShared) <= kNTiles * kNBytes, "the plan is made in the key ring before any copy");
constexpr uint32_t kTmS = 256, kTmP = 320, kTmQ = 352;
constexpr float kRescale = 8.0f;

struct UtShared {
  uint64_t nfull[kNTiles], nempty[kNTiles];
  uint64_t vfull[kVTiles], vempty[kVTiles];
  uint64_t qready, sfull, sfree, pfull, pvdone, ofree, done;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(UtShared) <= 512, "barrier block");

template <typename T>
__global__ void __launch_bounds__(kUtThreads, 1) paged_tc_kernel(const __grid_constant__ PagedParams p) {
  using E = Elem<T>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  UtShared* sh = reinterpret_cast<UtShared*>(smem + kUtBar);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int H = p.heads;
  volatile int* abort = &sh->abort;
  auto bar = [](uint64_t* b) { return smem_u32(b); };
  const int half = blockIdx.x & 1, w = blockIdx.x >> 1;

  PlanShared* plan = reinterpret_cast<PlanShared*>(smem + kUtN);
  grid_dep_launch_dependents();  // (the joining kernel may take its place)
  const long long total = plan_total(p, plan, kUtRows, blockIdx.x == 0);
  const int W = total > 0 ? plan_workers(total, p.workers) : 0;
  if (w >= W) {
    if (tid == 0) p.joins[w].rows = 0;
    return;
  }
  const long long x0 = plan_worker_begin(total, w, W), x1 = plan_worker_begin(total, w + 1, W);
  PlanCursor first;
  first.seek(p, plan, kUtRows, x0);

  if (tid == 0) {
    for (int i = 0; i < kNTiles; ++i) {
      mbar_init(bar(&sh->nfull[i]), kCopyWarps);
      mbar_init(bar(&sh->nempty[i]), 1);
    }
    for (int i = 0; i < kVTiles; ++i) {
      mbar_init(bar(&sh->vfull[i]), kCopyWarps);
      mbar_init(bar(&sh->vempty[i]), 1);
    }
    mbar_init(bar(&sh->qready), 4);
    mbar_init(bar(&sh->sfull), 1);
    mbar_init(bar(&sh->sfree), 4);
    mbar_init(bar(&sh->pfull), 4);
    mbar_init(bar(&sh->pvdone), 1);
    mbar_init(bar(&sh->ofree), 4);
    mbar_init(bar(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) tc::tmem_alloc(smem_u32(&sh->tmem), 512);
  // (the plan has been read: its place becomes the key ring)
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uniform(sh->tmem);

  // the key tiles [t0, t1) of an item that fall to this worker
  auto span = [&](const PlanCursor& c, int* t0, int* t1) {
    const int keys = c.q.keys_of_item(c.j, kUtRows, H);
    const int tiles = (keys + kKeyTile - 1) / kKeyTile;
    *t0 = c.tile_at(x0 > c.lo ? x0 : c.lo, tiles);
    *t1 = c.tile_at(x1 < c.hi ? x1 : c.hi, tiles);
    return keys;
  };

  if (warp == 4 || warp > 5) {
    // ============================================================ copies of key rows
    // A warp takes every third group of four keys; lanes 0-23 look up their cache rows.  Rows past the keys and of
    // bad blocks are zeros.  The values of the next tile are under way while a tile is completed.
    const int cw = warp == 4 ? 0 : warp - 5;
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t par) {
      ok = ok && at_wait_warp(bar(b), par, abort, p.budget_ns, p.status);
      return ok;
    };
    uint32_t un = 0, uv = 0, av = 0;  // stages filled, value stages announced
    PlanCursor c = first;
    for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kUtRows)) {
      int t0, t1;
      const int keys = span(c, &t0, &t1);
      auto rows_of = [&](int tile) {
        const int group = cw + kCopyWarps * (lane >> 2);
        const int k = tile * kKeyTile + group * 4 + (lane & 3);
        if (group >= kKeyTile / 4 || k >= keys || tile >= t1) return -1;
        const int pg = k / p.page;
        const int blk = p.table[(size_t)c.s * p.table_stride + pg];
        if (blk < 0 || blk >= p.nblocks) {
          atomicOr(p.status, kStatusBadSlot);
          return -1;
        }
        return blk * p.page + (k - pg * p.page);
      };
      // 64 columns x 4 blocks of every row, from block b0 of the latents: lane = 16-byte unit
      auto copy = [&](int rows, uint32_t base, int b0) {
        for (int i = 0; cw + kCopyWarps * i < kKeyTile / 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = __shfl_sync(~0u, rows, i * 4 + j);
            const int r = (cw + kCopyWarps * i) * 4 + j;
            const T* src = static_cast<const T*>(p.latent) + (size_t)max(row, 0) * p.lat_rs + b0 * 64 + lane * 8;
            cp_async16(base + (lane >> 3) * kBlk + r * 128 + (((lane & 7) ^ (r & 7)) * 16), src, row < 0 ? 0 : 16);
          }
      };
      auto values = [&](int rows) {
        const uint32_t s = uv % kVTiles;
        if (!wait(&sh->vempty[s], ((uv / kVTiles) & 1) ^ 1)) return;
        copy(rows, sbase + kUtV + s * kVBytes, half * 4);
        cp_async_commit();
        ++uv;
      };
      int row = rows_of(t0);
      if (t0 < t1) values(row);
      for (int t = t0; t < t1 && ok; ++t) {
        const int next = rows_of(t + 1);
        const uint32_t n = un % kNTiles;
        if (!wait(&sh->nempty[n], ((un / kNTiles) & 1) ^ 1)) break;
        const uint32_t base = sbase + kUtN + n * kNBytes;
        copy(row, base, (half ^ 1) * 4);
        for (int i = 0; cw + kCopyWarps * i < kKeyTile / 4; ++i) {  // k_pe: eight lanes a row
          const int kr = __shfl_sync(~0u, row, i * 4 + (lane >> 3));
          const int r = (cw + kCopyWarps * i) * 4 + (lane >> 3);
          const T* src = static_cast<const T*>(p.kpe) + (size_t)max(kr, 0) * p.kpe_rs + (lane & 7) * 8;
          cp_async16(base + 4 * kBlk + r * 128 + (((lane & 7) ^ (r & 7)) * 16), src, kr < 0 ? 0 : 16);
        }
        cp_async_commit();
        ++un;
        if (t + 1 < t1) {
          values(next);
          if (!ok) break;
          cp_async_wait<1>();
        } else {
          cp_async_wait<0>();
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(&sh->nfull[n]));
          mbar_arrive(bar(&sh->vfull[av % kVTiles]));
        }
        ++av;
        row = next;
      }
    }
    cp_async_wait<0>();
  } else if (warp == 5) {
    // ============================================================ MMA (one thread)
    if (tc::elect_one()) {
      const uint32_t id_qk = tc::idesc_f16(E::kBf16, 128, 64, false, false);
      const uint32_t id_pv = tc::idesc_f16(E::kBf16, 128, 256, false, true);
      const uint64_t dn = tc::sdesc_sw128(sbase + kUtN, 16, 1024), dq = tc::sdesc_sw128(sbase + kUtQ, 16, 1024);
      const uint64_t dvk = tc::sdesc_sw128(sbase + kUtV, 16, 1024), dv = tc::sdesc_sw128(sbase + kUtV, kBlk, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t par) {
        ok = ok && at_wait(bar(b), par, abort, p.budget_ns, p.status);
        return ok;
      };
      uint32_t ns = 0, np = 0, ks = 0, kp = 0, vs = 0;  // stages (and phases) of the rings
      uint32_t g_qk = 0, g_pv = 0, item = 0;
      auto qk = [&]() {  // scores of tile g_qk
        if (!wait(&sh->sfree, (g_qk & 1) ^ 1) || !wait(&sh->nfull[ns], np)) return;
        tc::fence_after_sync();
        const uint64_t bn = dn + ns * (kNBytes >> 4);
#pragma unroll
        for (int k = 0; k < 20; ++k)
          tc::mma_f16_ts(tmem + kTmS, tmem + kTmQ + k * 8, bn + (k >> 2) * (kBlk >> 4) + 2 * (k & 3), id_qk, k > 0);
        tc::commit(bar(&sh->nempty[ns]));
        if (++ns == kNTiles) {
          ns = 0;
          np ^= 1;
        }
        if (!wait(&sh->vfull[ks], kp)) return;
        const uint64_t bv = dvk + ks * (kVBytes >> 4);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          tc::mma_f16(tmem + kTmS, dq + (k >> 2) * (16384 >> 4) + 2 * (k & 3), bv + (k >> 2) * (kBlk >> 4) + 2 * (k & 3), id_qk, true);
        tc::commit(bar(&sh->sfull));
        if (++ks == kVTiles) {
          ks = 0;
          kp ^= 1;
        }
        ++g_qk;
      };
      PlanCursor c = first;
      for (bool more = true; more && c.lo < x1 && ok; more = c.next(p, kUtRows)) {
        int t0, t1;
        span(c, &t0, &t1);
        if (t0 >= t1) continue;
        if (!wait(&sh->qready, item & 1)) break;
        tc::fence_after_sync();
        qk();
        for (int t = t0; t < t1 && ok; ++t) {
          if (t + 1 < t1) qk();
          if (!ok) break;
          // output of tile t
          if (t == t0 && item > 0 && !wait(&sh->ofree, (item - 1) & 1)) break;
          if (!wait(&sh->pfull, g_pv & 1)) break;
          tc::fence_after_sync();
          const uint64_t bd = dv + vs * (kVBytes >> 4);
          tc::mma_f16_ts(tmem, tmem + kTmP, bd, id_pv, t > t0);
#pragma unroll
          for (int k = 1; k < 4; ++k) tc::mma_f16_ts(tmem, tmem + kTmP + k * 8, bd + k * 128, id_pv, true);
          tc::commit(bar(&sh->vempty[vs]));
          tc::commit(bar(&sh->pvdone));
          if (++vs == kVTiles) vs = 0;
          ++g_pv;
        }
        ++item;
      }
      // every MMA issued so far has completed before TMEM is released
      tc::commit(bar(&sh->done));
      mbar_wait_bounded(bar(&sh->done), 0, drain_budget(p.budget_ns));
    }
    __syncwarp();
  } else {
    // ============================================================ queries, softmax, results
    const int r = tid;  // row of the item
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float scale = p.scale_log2;
    uint32_t g = 0;  // tiles done
    bool ok = true;
    auto arrive = [&](uint64_t* b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    auto load_q = [&](const PlanCursor& c) {
      const int row = c.j * kUtRows + r;
      const bool live = row < c.q.n * H;
      const int tok = live ? row / H : 0, hd = live ? row - tok * H : 0;
      const uint4* ql = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q_lat) + (size_t)(c.q.begin + tok) * p.ql_ts + (size_t)hd * p.ql_hs);
      const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q_pe) + (size_t)(c.q.begin + tok) * p.qp_ts + (size_t)hd * p.qp_hs);
#pragma unroll 3
      for (int j = 0; j < 9; ++j) {  // the score-only blocks' columns, then this half's
        const uint4* src = j < 4 ? ql + ((half ^ 1) * 4 + j) * 8 : j == 4 ? qp : ql + (half * 4 + j - 5) * 8;
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
        if (j < 5) {
          tc::st16(tmem + lanes + kTmQ + j * 32, reinterpret_cast<const uint32_t*>(v));
          tc::st16(tmem + lanes + kTmQ + j * 32 + 16, reinterpret_cast<const uint32_t*>(v + 4));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(smem + kUtQ + (j - 5) * 16384 + r * 128 + ((i ^ (r & 7)) * 16)) = v[i];
        }
      }
      tc::wait_st();
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      arrive(&sh->qready);
    };
    PlanCursor c = first;
    {
      int t0, t1;
      span(c, &t0, &t1);
      if (t0 < t1) load_q(c);
    }
    for (bool more = true; more && c.lo < x1 && ok;) {
      int t0, t1;
      const int keys = span(c, &t0, &t1);
      if (tid == 0 && half == 0 && c.hi >= x1) plan_post_join(p, c, kUtRows, w, x0, x1, total, W);
      const int row = c.j * kUtRows + r;
      const bool live = row < c.q.n * H;
      const int limit0 = live ? c.q.keys_of_row(row, H) : 0;
      const bool whole = c.lo >= x0 && c.hi <= x1;
      const size_t grow = (size_t)c.q.begin * H + row;
      const size_t slot = (size_t)w * 2 + (c.lo < x0 ? 0 : 1);
      float m = -INFINITY, l = 0.f;
      for (int t = t0; t < t1; ++t, ++g) {
        if (!at_wait_warp(bar(&sh->sfull), g & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
        tc::fence_after_sync();
        uint32_t s[64];
        tc::ld32(tmem + lanes + kTmS, s);
        tc::ld32(tmem + lanes + kTmS + 32, s + 32);
        tc::wait_ld();
        tc::fence_before_sync();
        arrive(&sh->sfree);
        const int limit = limit0 - t * kKeyTile;
        if (__any_sync(~0u, limit < kKeyTile)) {
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
        const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        float f = 1.f;
        const bool grow_max = __any_sync(~0u, (tile_max - m) * scale > kRescale);
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
        if (grow_max && t > t0) tmem_scale<256>(tmem + lanes, f);
        tc::st16(tmem + lanes + kTmP, pk);
        tc::st16(tmem + lanes + kTmP + 16, pk + 16);
        tc::wait_st();
        tc::fence_before_sync();
        const int valid = keys - t * kKeyTile;
        if (valid < kKeyTile) {
          // latents past the keys: whole 128-byte rows, so the swizzle does not matter (the scores of this tile,
          // which read them too, are done)
          for (int x = tid; x < (kKeyTile - valid) * 32; x += 128)
            *reinterpret_cast<uint4*>(smem + kUtV + (g % kVTiles) * kVBytes + ((x >> 3) & 3) * kBlk + (valid + x / 32) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
        }
        arrive(&sh->pfull);
      }
      if (!ok) break;
      // the next item's queries go in while the last output MMA runs
      more = c.next(p, kUtRows);
      if (more && c.lo < x1) {
        int u0, u1;
        span(c, &u0, &u1);
        if (u0 < u1) load_q(c);
      }
      if (t0 < t1) {
        if (!at_wait_warp(bar(&sh->pvdone), (g - 1) & 1, abort, p.budget_ns, p.status)) { ok = false; break; }
        tc::fence_after_sync();
      }
      const float iv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      T* out = static_cast<T*>(p.out) + (live ? grow : 0) * kRank + half * 256;
      float* po = p.part_o + (slot * kUtRows + r) * kRank + half * 256;
      if (t0 < t1) {
#pragma unroll 1
        for (int cc = 0; cc < 256; cc += 32) {
          uint32_t o[32];
          tc::ld32(tmem + lanes + cc, o);
          tc::wait_ld();
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t q[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                q[j] = E::pack(__uint_as_float(o[k + 2 * j]) * iv, __uint_as_float(o[k + 2 * j + 1]) * iv);
              *reinterpret_cast<uint4*>(out + cc + k) = make_uint4(q[0], q[1], q[2], q[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(po + cc + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        tc::fence_before_sync();
        arrive(&sh->ofree);
      } else if (whole && live) {  // no key at all
        for (int cc = 0; cc < 256; cc += 8) *reinterpret_cast<uint4*>(out + cc) = make_uint4(0, 0, 0, 0);
      }
      if (half == 0 && live) {
        if (!whole) {
          float* ml = p.part_ml + (slot * kUtRows + r) * 2;
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
  if (warp == 5) tc::tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t paged_tc_prepare(bool bf16) {
  return bf16 ? cudaFuncSetAttribute(paged_tc_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kUtSmem)
              : cudaFuncSetAttribute(paged_tc_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kUtSmem);
}

cudaError_t paged_tc_launch(bool bf16, const PagedParams& p, cudaStream_t stream) {
  if (bf16)
    paged_tc_kernel<__nv_bfloat16><<<p.workers * 2, kUtThreads, kUtSmem, stream>>>(p);
  else
    paged_tc_kernel<__half><<<p.workers * 2, kUtThreads, kUtSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
