// paged_kv_plan.cuh -- how the paged K/V attention shares its work.
//
// The split of paged_plan.cuh with one more level: an item is (sequence, KV
// head, block of R consecutive query rows), a query row a (token, head of the
// group) pair, row = token * G + g.  All KV heads of a sequence cost the same,
// so a sequence is KH times the cost of one head.  Workers are warps; keys
// are counted in tiles of kKvTile.
#pragma once
#include "paged_plan.cuh"

namespace mla {

constexpr int kKvTile = 32;

__host__ __device__ __forceinline__ Seq kv_seq(const PagedKvParams& p, int s, int R, bool report) {
  Seq q = plan_seq(p.plan, s, R, report);
  q.first = q.last = p.item_cost;
  if (q.items > 0) {
    q.first += (q.keys_of_item(0, R, p.plan.heads) + kKvTile - 1) / kKvTile;
    q.last += (q.keys_of_item(q.items - 1, R, p.plan.heads) + kKvTile - 1) / kKvTile;
  }
  return q;
}

// Cost of all sequences; ps->base[i] = cost before thread i's strip.
__device__ __forceinline__ long long kv_total(const PagedKvParams& p, PlanShared* ps, int R, bool report) {
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int strip = (p.plan.nseq + nt - 1) / nt;
  long long mine = 0;
  for (int i = 0; i < strip; ++i) {
    const int s = tid * strip + i;
    if (s < p.plan.nseq) {
      const Seq q = kv_seq(p, s, R, report);
      mine += q.cum(q.items) * p.kv_heads;
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
  long long before = 0, all = 0;
  for (int w = 0; w < nt / 32; ++w) {
    const long long x = ps->warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  ps->base[tid] = before + inc - mine;
  if (tid == 0) {
    ps->base[nt] = all;
    ps->threads = nt;
  }
  __syncthreads();
  return all;
}

// Workers that take part, at least kKvMinRange of cost each.
constexpr int kKvMinRange = 1;
__host__ __device__ __forceinline__ int kv_workers(long long total, int W) {
  const long long w = total / kKvMinRange;
  return w < 1 ? 1 : (w < W ? (int)w : W);
}

// A place in the list of items: sequence, KV head, item, and the item's cost range.
struct KvCursor {
  int s, head, j, own;  // (own: item_cost)
  Seq q;
  long long seq_base, head_cost;
  long long lo, hi;

  __host__ __device__ __forceinline__ void set(int h, int jj) {
    head = h;
    j = jj;
    const long long base = seq_base + h * head_cost;
    lo = base + q.cum(jj);
    hi = base + q.cum(jj + 1);
  }
  __host__ __device__ __forceinline__ void open(const PagedKvParams& p, int ss, int R) {
    s = ss;
    own = p.item_cost;
    q = kv_seq(p, ss, R, false);
    head_cost = q.cum(q.items);
  }
  // The item that holds position x (0 <= x < total).
  __host__ __device__ __forceinline__ void seek(const PagedKvParams& p, const PlanShared* ps, int R, long long x) {
    const int nt = ps->threads;
    const int strip = (p.plan.nseq + nt - 1) / nt;
    int a = 0, b = nt;  // last strip with base <= x
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (ps->base[m] <= x) a = m; else b = m;
    }
    seq_base = ps->base[a];
    open(p, a * strip, R);
    while (seq_base + head_cost * p.kv_heads <= x) {
      seq_base += head_cost * p.kv_heads;
      open(p, s + 1, R);
    }
    const int h = (int)((x - seq_base) / head_cost);
    const long long base = seq_base + h * head_cost;
    int l = 0, hh = q.items;
    while (hh - l > 1) {
      const int m = (l + hh) / 2;
      if (base + q.cum(m) <= x) l = m; else hh = m;
    }
    set(h, l);
  }
  // The next item; false past the last one.
  __host__ __device__ __forceinline__ bool next(const PagedKvParams& p, int R) {
    if (j + 1 < q.items) {
      set(head, j + 1);
      return true;
    }
    if (head + 1 < p.kv_heads) {
      set(head + 1, 0);
      return true;
    }
    do {
      seq_base += head_cost * p.kv_heads;
      if (s + 1 >= p.plan.nseq) return false;
      open(p, s + 1, R);
    } while (q.items == 0);
    set(0, 0);
    return true;
  }
  // Key tile that position x of this item (lo <= x <= hi) stands for.
  __host__ __device__ __forceinline__ int tile_at(long long x, int tiles) const {
    const long long d = hi - lo - own;
    if (d < 1) return x < hi ? 0 : tiles;
    const long long y = x - lo - own;
    if (y <= 0) return 0;
    const long long n = y * tiles;
    return n < (1ll << 31) ? (int)((uint32_t)n / (uint32_t)d) : (int)(n / d);
  }
};

// Worker w's record for the joining kernel, made at the last item of its
// range (PagedJoin: `row` counts token * G + g, `pad` is the KV head).
__host__ __device__ __forceinline__ void kv_post_join(const PagedKvParams& p, const KvCursor& c, int R, int w, long long x0,
                                                      long long x1, long long total, int W) {
  PagedJoin j = {0, 0, 0, 0};
  if (c.lo >= x0 && c.hi > x1) {
    const int G = p.plan.heads, left = c.q.n * G - c.j * R;
    j.row = c.q.begin * G + c.j * R;
    j.rows = left < R ? left : R;
    j.last_worker = plan_worker_of(c.hi - 1, total, W);
    j.pad = c.head;
  }
  p.plan.joins[w] = j;
}

// The workers that an item is split over, seen from worker w with the range
// [x0, x1): the first and the last.
__host__ __device__ __forceinline__ void kv_sharers(const KvCursor& c, int w, long long x0, long long x1, long long total, int W,
                                                    int* first, int* last) {
  *first = c.lo >= x0 ? w : plan_worker_of(c.lo, total, W);
  *last = c.hi <= x1 ? w : plan_worker_of(c.hi - 1, total, W);
}

}  // namespace mla
