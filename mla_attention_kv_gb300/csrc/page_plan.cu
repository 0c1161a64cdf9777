// page_plan.cu -- one step's plan of a paged cache, made on the device from
// the requests' lengths: pages of sequences that end go back to the stack of
// free blocks, pages for new tokens come from it, and every token row gets
// its cache slot and its position.
//
// Sequence i with L cached and n new tokens (an ended one: L = 0):
//   need_i = max(0, ceil((L + n) / page) - h),  k_i = sum_{j<i} need_j
//   its m-th new page is free[count - 1 - (k_i + m)]
// h being the pages it holds: ceil(L / page), or where the caller keeps counts
// (sequences that become shorter when drafted tokens are rejected) its count.
//   row cu_q[i] + j: position L + j, slot = block * page + position % page
// Two prefix sums over the sequences, then one thread per row and per page
// that finds its sequence by bisection.  Every order is fixed, so the result
// does not depend on timing.
//
// A few KB per step: all latency.  One cluster works on it; each of its CTAs
// makes the prefix sums by itself (the inputs come from L2 after the first)
// and takes its share of the rows and pages, so that the only exchanges are
// the cluster barriers that keep reads of the inputs before the writes of
// the outputs that may share their memory (lengths, count, table, stack).
#include "attn.h"
#include "common.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kPlThreads = 512;
constexpr int kPlUnroll = 4;  // pages of a thread in flight

struct PlShared {
  long long warp_sum[2][kPlThreads / 32];
  int begin[kPlThreads + 1];  // first token row of each sequence of the strip
  int k[kPlThreads + 1];      // pages handed out before it (or, in the first pass, taken back)
  int old[kPlThreads];        // cached tokens
  int first[kPlThreads];      // pages it held
  int ok[kPlThreads];
  int used;
};

// Exclusive prefix sum over the block; *total gets the sum.
__device__ __forceinline__ long long pl_scan(PlShared& sh, int which, long long v, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) sh.warp_sum[which][warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const long long x = sh.warp_sum[which][w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + inc - v;
}

// The last i of a[0 .. n) with a[i] <= x (a[0] <= x, a not decreasing).
__device__ __forceinline__ int pl_find(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlThreads) page_plan_kernel(const PagePlanParams p) {
  __shared__ PlShared sh;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int rank = blockIdx.x, ctas = gridDim.x;  // (the grid is one cluster)
  const int me = rank * nt + tid, all = ctas * nt;
  const long long width = (long long)p.table_stride * p.page;
  const int cap = width < kMaxSeqTokens ? (int)width : kMaxSeqTokens;
  unsigned bad = 0;

  int count = *p.free_count;
  if (count < 0 || count > p.nblocks) {
    bad |= kStatusBadLength;
    count = count < 0 ? 0 : p.nblocks;
  }
  auto cached = [&](int i) {  // tokens in the cache before the step
    int L = p.kv_lens[i];
    if (L < 0 || L > cap) {
      bad |= kStatusBadLength;
      L = L < 0 ? 0 : cap;
    }
    return L;
  };
  auto pages = [&](int L) { return (int)(((unsigned)L + p.page - 1) / (unsigned)p.page); };
  auto holds = [&](int i, int L) {  // pages of sequence i with L cached tokens
    const int own = pages(L);
    if (!p.held) return own;
    int h = p.held[i];
    if (h < own || h > p.table_stride) {
      bad |= kStatusBadLength;
      h = h < own ? own : p.table_stride;
    }
    return h;
  };

  // ---- pages of the sequences that end, in (sequence, page) order onto the stack
  if (p.ended) {
    long long back = 0;
    for (int s0 = 0; s0 < p.nseq; s0 += nt) {
      const int i = s0 + tid;
      const int give = i < p.nseq && p.ended[i] ? holds(i, cached(i)) : 0;
      long long total;
      const long long at = pl_scan(sh, 0, give, &total);
      if (total > 0) {  // (the same for all threads)
        const int most = (int)(total < p.nblocks ? total : p.nblocks);
        sh.k[tid] = at < p.nblocks ? (int)at : p.nblocks;
        __syncthreads();
        const int live = min(nt, p.nseq - s0);
        if (total > most || count + back + total > p.nblocks) bad |= kStatusBadLength;
        for (int x0 = me; x0 < most; x0 += kPlUnroll * all) {
          int v[kPlUnroll];
#pragma unroll
          for (int i = 0; i < kPlUnroll; ++i) {
            const int x = x0 + i * all;
            if (x >= most) break;
            // (sequences that give none share their k with the next one that gives)
            const int q = pl_find(sh.k, live, x);
            v[i] = p.table[(size_t)(s0 + q) * p.table_stride + (x - sh.k[q])];
          }
#pragma unroll
          for (int i = 0; i < kPlUnroll; ++i) {
            const long long to = count + back + x0 + i * all;
            if (x0 + i * all < most && to < p.nblocks) p.free_blocks[to] = v[i];
          }
        }
      }
      back += total;
      __syncthreads();
    }
    count = (int)(count + back < p.nblocks ? count + back : p.nblocks);
    if (ctas > 1) tc::cluster_sync(); else __syncthreads();  // the stack is complete (and the table read)
  }

  // ---- the step's tokens and pages, a strip of sequences at a time
  long long row0 = 0, page0 = 0;  // rows and pages before the strip
  int used = 0;
  for (int s0 = 0; s0 < p.nseq || s0 == 0; s0 += nt) {
    const int i = s0 + tid;
    const int live = min(nt, p.nseq - s0);
    int n = 0, L = 0, first = 0;
    bool ok = false;
    if (i < p.nseq) {
      n = p.new_lens[i];
      if (n < 0) {
        bad |= kStatusBadLength;
        n = 0;
      }
      if (!p.ended || !p.ended[i]) {
        L = cached(i);
        first = holds(i, L);
      }
    }
    long long rows, need_all;
    const long long at = row0 + pl_scan(sh, 0, n, &rows);
    const long long end = at + n;
    if (i < p.nseq) {
      ok = end <= p.T && (long long)L + n <= cap;
      if (!ok) bad |= kStatusBadLength;
    }
    const int need = ok ? max(0, pages(L + n) - first) : 0;
    const long long k = page0 + pl_scan(sh, 1, need, &need_all);
    if (ok && need > 0 && k + need > count) {
      ok = false;
      bad |= kStatusNoPages;
    }
    sh.begin[tid] = (int)(at < p.T ? at : p.T);
    sh.k[tid] = (int)(k < p.nblocks ? k : p.nblocks);
    sh.old[tid] = L;
    sh.first[tid] = first;
    sh.ok[tid] = ok;
    if (tid == 0) sh.used = used;
    // every CTA has read the strip's lengths (the second scan has read the first one's sums)
    if (ctas > 1) tc::cluster_sync(); else __syncthreads();
    if (ok && need > 0) atomicMax(&sh.used, (int)(k + need));
    if (rank == 0 && i < p.nseq) {
      p.kv_lens_out[i] = ok ? L + n : L;
      if (p.held) p.held_out[i] = ok ? first + need : first;
      if (i == 0) p.cu_q[0] = 0;
      p.cu_q[i + 1] = (int)(end < p.T ? end : p.T);
    }
    const int lo = (int)(row0 < p.T ? row0 : p.T), hi = (int)(row0 + rows < p.T ? row0 + rows : p.T);
    for (int r = lo + me; r < hi; r += all) {
      const int q = pl_find(sh.begin, live, r);
      int slot = -1, pos = 0;
      if (sh.ok[q]) {
        pos = sh.old[q] + r - sh.begin[q];
        const int pg = (int)((unsigned)pos / (unsigned)p.page), m = pg - sh.first[q];
        const int blk = m >= 0 ? p.free_blocks[count - 1 - (sh.k[q] + m)] : p.table[(size_t)(s0 + q) * p.table_stride + pg];
        if (blk >= 0 && blk < p.nblocks)
          slot = blk * p.page + pos - pg * p.page;
        else
          bad |= kStatusBadSlot;
      }
      p.slots[r] = slot;
      p.positions[r] = pos;
    }
    const int plo = (int)(page0 < count ? page0 : count), phi = (int)(page0 + need_all < count ? page0 + need_all : count);
    for (int x = plo + me; x < phi; x += all) {
      const int q = pl_find(sh.k, live, x);
      if (sh.ok[q]) p.table[(size_t)(s0 + q) * p.table_stride + sh.first[q] + x - sh.k[q]] = p.free_blocks[count - 1 - x];
    }
    row0 += rows;
    page0 += need_all;
    __syncthreads();
    used = sh.used;
    __syncthreads();
  }
  if (rank == 0 && tid == 0) {
    *p.free_count_out = count - used;
    if (p.nseq == 0) p.cu_q[0] = 0;
  }
  for (long long r = (row0 < p.T ? row0 : p.T) + me; r < p.T; r += all) {  // rows of no sequence
    p.slots[r] = -1;
    p.positions[r] = 0;
  }
  if (bad) atomicOr(p.status, bad);
}

}  // namespace

cudaError_t page_plan_launch(const PagePlanParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t c = {};
  // One CTA while a few passes of its threads do; the pages that come back are
  // known on the device only, so the table's size stands for them.  64
  // sequences, one token each: 4.8 us on one CTA, 5.5 on eight; 256 sequences with 16384 rows: 20.1 and 8.7.
  const long long pages = p.ended ? (long long)p.nseq * p.table_stride : 0;
  const int ctas = p.T <= 4 * kPlThreads && pages <= 16 * kPlThreads ? 1 : 8;
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kPlThreads);
  c.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, page_plan_kernel, p);
}

}  // namespace mla
