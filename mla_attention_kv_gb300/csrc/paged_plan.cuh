// paged_plan.cuh -- how the paged attention kernels share their work.
//
// A work item is (sequence, block of R consecutive query rows); a query row
// is a (token, head) pair, row = token * H + head.  Its keys are taken in
// tiles of kKeyTile.  The lengths live on the device, so the split is made
// there: every item gets a width in a common cost space (about its number of
// key tiles, plus a constant for what an item costs by itself), the widths
// of all items are laid end to end, and worker w of W takes the cost range
// [total * w / W, total * (w + 1) / W).  A range may begin and end inside an
// item; such items are computed in pieces whose results (unnormalised
// output, maximum, sum) go to the workspace and are joined in a fixed order
// by the combine kernel, so results do not depend on timing.
//
// The cumulative cost inside a sequence is the closed form
//   F(j) = j * first + (last - first) * j^2 / (2 * items),
// first / last being the widths of its first and last item (the causal limit
// grows along the chunk): exact for one item, an even slope for many.  A
// position x inside item j is mapped to the key tile
// (x - F(j) - cost) * tiles / (width - cost), by both neighbours alike.
#pragma once
#include <stdint.h>

#include "attn.h"
#include "common.cuh"

namespace mla {

constexpr int kKeyTile = 64;
// Width of an item beyond its key tiles (loading its queries, storing its
// result), in key tiles.  128-row items: about 10 us for 0.95 us a key tile
// (32 sequences of 100 to 2000 keys, 128 heads: 47 us at cost 1, 33 at 10).
// It stands before the item's first key tile, so that a worker that begins an
// item pays for it and one that goes on with it does not (4 sequences of 20000
// to 32768 keys, 2 tokens of 128 heads: 66 us, 71 with the cost spread over the
// item's tiles).
__host__ __device__ constexpr int plan_item_cost(int R) { return R == kPagedPairRows ? 10 : 1; }
constexpr int kPlanThreadsMax = 512;
// Longest sequence: a tile beyond its last one still has key numbers of 31 bits.
constexpr int kMaxKeys = 0x7fffff00;

struct PlanShared {
  int threads;
  long long base[kPlanThreadsMax + 1];  // cost before each thread's strip of sequences
  long long warp_sum[kPlanThreadsMax / 32];
};

struct Seq {
  int begin;  // first token row
  int n;      // new tokens
  int L;      // cached tokens (the new ones included)
  int items;
  int first, last;  // widths of the first and last item

  __host__ __device__ __forceinline__ int keys_of_row(int row_in_seq, int H) const {
    const int t = row_in_seq / H;
    const int k = L - n + t + 1;
    return k < 0 ? 0 : (k > L ? L : k);
  }
  // keys of item j: those of its last row
  __host__ __device__ __forceinline__ int keys_of_item(int j, int R, int H) const {
    const long long last_row = (long long)(j + 1) * R - 1;
    const long long rows = (long long)n * H;
    return keys_of_row((int)(last_row < rows ? last_row : rows - 1), H);
  }
  __host__ __device__ __forceinline__ long long cum(int j) const {
    if (last == first) return (long long)j * first;  // (decode: no division)
    // (the divisor of a sequence without items only has to be nonzero)
    return (long long)j * first + (long long)(last - first) * j * j / (2 * (long long)(items > 0 ? items : 1));
  }
};

// Sequence s of the call.  Lengths out of range are clamped and, where
// `report`, recorded.
__host__ __device__ __forceinline__ Seq plan_seq(const PagedParams& p, int s, int R, bool report) {
  Seq q;
  bool bad = false;
  if (p.cu_q) {
    int a = p.cu_q[s], b = p.cu_q[s + 1];
    if (a < 0 || a > p.T) { bad = true; a = a < 0 ? 0 : p.T; }
    if (b < a || b > p.T) { bad = true; b = b < a ? a : p.T; }
    q.begin = a;
    q.n = b - a;
  } else {
    q.begin = s * p.n_uniform;
    q.n = p.n_uniform;
  }
  const long long width = (long long)p.table_stride * p.page, cap = width < kMaxKeys ? width : kMaxKeys;
  int L = p.kv_lens[s];
  if (L < 0) { bad = true; L = 0; }
  if (L > cap) { bad = true; L = (int)cap; }
  q.L = L;
  const long long rows = (long long)q.n * p.heads;
  q.items = (int)((rows + R - 1) / R);
  q.first = q.last = plan_item_cost(R);
  if (q.items > 0) {
    q.first += (q.keys_of_item(0, R, p.heads) + kKeyTile - 1) / kKeyTile;
    q.last += (q.keys_of_item(q.items - 1, R, p.heads) + kKeyTile - 1) / kKeyTile;
  }
#ifdef __CUDA_ARCH__
  if (report && bad) atomicOr(p.status, kStatusBadLength);
#endif
  return q;
}

// Cost of all sequences; ps->base[i] = cost before thread i's strip.  All
// threads of the block (a multiple of 32, at most kPlanThreadsMax).
__device__ __forceinline__ long long plan_total(const PagedParams& p, PlanShared* ps, int R, bool report) {
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int strip = (p.nseq + nt - 1) / nt;
  long long mine = 0;
  for (int i = 0; i < strip; ++i) {
    const int s = tid * strip + i;
    if (s < p.nseq) {
      const Seq q = plan_seq(p, s, R, report);
      mine += q.cum(q.items);
    }
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) ps->warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < warp; ++w) before += ps->warp_sum[w];
  ps->base[tid] = before + inc - mine;
  if (tid == nt - 1) {
    ps->base[nt] = before + inc;
    ps->threads = nt;
  }
  __syncthreads();
  return ps->base[nt];
}

// Workers that take part: no range is shorter than this.  16-row items: 2
// instead of 1 took one sequence of 777 tokens from 15.6 to 16.5 us.  128-row
// items: one sequence of 4096 keys 30.4 us at 1, 26.7 at 2, 24.8 at 3; eight of
// 500 to 3000 keys 26.6 us up to 3, 33.8 at 4.
__host__ __device__ constexpr int plan_min_range(int R) { return R == kPagedPairRows ? 3 : 1; }
__host__ __device__ __forceinline__ int plan_workers(long long total, int W, int R) {
  const long long w = total / plan_min_range(R);
  return w < 1 ? 1 : (w < W ? (int)w : W);
}
__host__ __device__ __forceinline__ long long plan_worker_begin(long long total, int w, int W) {
  const long long n = total * w;
  return n < (1ll << 32) ? (uint32_t)n / (uint32_t)W : n / W;
}
// The worker whose range holds position x.
__host__ __device__ __forceinline__ int plan_worker_of(long long x, long long total, int W) {
  const long long n = (x + 1) * W - 1;
  return n < (1ll << 32) && total < (1ll << 32) ? (int)((uint32_t)n / (uint32_t)total) : (int)(n / total);
}

// A place in the list of items: sequence, item, and the item's cost range.
struct PlanCursor {
  int s;
  Seq q;
  long long seq_base;
  int j;
  long long lo, hi;

  __host__ __device__ __forceinline__ void set_item(int jj) {
    j = jj;
    lo = seq_base + q.cum(jj);
    hi = seq_base + q.cum(jj + 1);
  }
  // The item that holds position x (0 <= x < total).
  __host__ __device__ __forceinline__ void seek(const PagedParams& p, const PlanShared* ps, int R, long long x) {
    const int nt = ps->threads;
    const int strip = (p.nseq + nt - 1) / nt;
    int a = 0, b = nt;  // last strip with base <= x
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (ps->base[m] <= x) a = m; else b = m;
    }
    s = a * strip;
    seq_base = ps->base[a];
    q = plan_seq(p, s, R, false);
    while (seq_base + q.cum(q.items) <= x) {
      seq_base += q.cum(q.items);
      ++s;
      q = plan_seq(p, s, R, false);
    }
    int l = 0, h = q.items;
    while (h - l > 1) {
      const int m = (l + h) / 2;
      if (seq_base + q.cum(m) <= x) l = m; else h = m;
    }
    set_item(l);
  }
  // The next item; false past the last one.
  __host__ __device__ __forceinline__ bool next(const PagedParams& p, int R) {
    if (j + 1 < q.items) {
      set_item(j + 1);
      return true;
    }
    do {
      seq_base += q.cum(q.items);
      if (++s >= p.nseq) return false;
      q = plan_seq(p, s, R, false);
    } while (q.items == 0);
    set_item(0);
    return true;
  }
  // Key tile that position x of this item (lo <= x <= hi) stands for.
  __host__ __device__ __forceinline__ int tile_at(long long x, int tiles, int R) const {
    const long long d = hi - lo - plan_item_cost(R);
    if (d < 1) return x < hi ? 0 : tiles;
    const long long y = x - lo - plan_item_cost(R);
    if (y <= 0) return 0;
    const long long n = y * tiles;
    return n < (1u << 31) ? (int)((uint32_t)n / (uint32_t)d) : (int)(n / d);
  }
};

// The joining kernel runs whatever becomes of the workers, so a worker's
// record is empty from before its first wait until plan_post_join: a worker
// that gives up leaves nothing for it to do, and never what an earlier call
// of the handle (perhaps a larger one) has left there.  The thread that posts.
__host__ __device__ __forceinline__ void plan_open_join(const PagedParams& p, int w) { p.joins[w] = PagedJoin{0, 0, 0, 0}; }

// Whether a record of worker w1 stays within this call's rows and workers.
// Posted ones do, unless the lengths changed while the call ran and its
// workers saw different ones.
__host__ __device__ __forceinline__ bool plan_join_fits(const PagedParams& p, const PagedJoin& j, int w1, int R) {
  return j.row >= 0 && j.rows >= 0 && j.rows <= R && (long long)j.row + j.rows <= (long long)p.T * p.heads &&
         j.last_worker >= w1 && j.last_worker < p.workers;
}

// Worker w's record for the joining kernel, made at the last item of its
// range: the rows of that item if the item begins with it and goes on with
// others.  One thread.
__host__ __device__ __forceinline__ void plan_post_join(const PagedParams& p, const PlanCursor& c, int R, int w, long long x0,
                                                        long long x1, long long total, int W) {
  PagedJoin j = {0, 0, 0, 0};
  if (c.lo >= x0 && c.hi > x1) {
    const int left = c.q.n * p.heads - c.j * R;
    j.row = c.q.begin * p.heads + c.j * R;
    j.rows = left < R ? left : R;
    j.last_worker = plan_worker_of(c.hi - 1, total, W);
  }
  p.joins[w] = j;
}

}  // namespace mla
