// prompt_plan.cuh -- which query block of which sequence and head a CTA of
// the prompt attention works on.
//
// Items are (head, block of query rows of a sequence), head after head, so
// that the CTAs at work share few heads' keys in L2; the blocks of a
// sequence are taken from its end, where a causal block has the most keys.
// CTA c of C takes items c, 2C - 1 - c, 2C + c, 4C - 1 - c, ...: the
// direction alternates so that no CTA always gets the longer blocks.
#pragma once
#include "attn.h"
#include "common.cuh"

namespace mla {

constexpr int kPromptPlanThreads = 320;

struct PromptPlace {
  int batch, begin, len, row0;  // sequence: rows begin .. begin + len of `batch`; first query row in it
  int head;
};

struct PromptPlan {
  int base[kPromptPlanThreads + 1];  // packed: blocks before each thread's strip of sequences
  int warp_sum[32];
};

// Length of packed sequence i, clamped to the s rows there are.
__device__ __forceinline__ int prompt_seq(const PromptParams& p, int i, int* begin, bool report) {
  int a = p.cu[i], b = p.cu[i + 1];
  bool bad = false;
  if (a < 0 || a > p.s) { bad = true; a = a < 0 ? 0 : p.s; }
  if (b < a || b > p.s) { bad = true; b = b < a ? a : p.s; }
  if (report && bad) atomicOr(p.status, kStatusBadLength);
  *begin = a;
  return b - a;
}

// Number of query blocks (of `rows` rows) per head; all threads of a block
// of kPromptPlanThreads.
__device__ __forceinline__ int prompt_plan(const PromptParams& p, PromptPlan* ps, int rows, bool report) {
  if (!p.cu) return (p.s + rows - 1) / rows * p.b;
  const int nt = kPromptPlanThreads, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int strip = (p.nseq + nt - 1) / nt;
  int mine = 0, begin;
  for (int i = 0; i < strip; ++i)
    if (tid * strip + i < p.nseq) mine += (prompt_seq(p, tid * strip + i, &begin, report) + rows - 1) / rows;
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) ps->warp_sum[warp] = inc;
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < warp; ++w) before += ps->warp_sum[w];
  ps->base[tid] = before;
  if (tid == nt - 1) ps->base[nt] = before + mine;
  __syncthreads();
  return ps->base[nt];
}

// Item of CTA c of C in its k-th round.
__device__ __forceinline__ long long prompt_item(int c, int C, int k) {
  return (long long)k * C + ((k & 1) ? C - 1 - c : c);
}

// Place of item x (of blocks * heads); any thread by itself.
__device__ __forceinline__ PromptPlace prompt_place(const PromptParams& p, const PromptPlan* ps, long long x, int blocks, int rows) {
  PromptPlace r;
  r.head = (int)(x / blocks);
  int i = (int)(x - (long long)r.head * blocks);
  if (!p.cu) {
    const int per = (p.s + rows - 1) / rows;
    r.batch = i / per;
    r.begin = 0;
    r.len = p.s;
    r.row0 = (per - 1 - (i - r.batch * per)) * rows;
    return r;
  }
  int a = 0, b = kPromptPlanThreads;  // last strip with base <= i
  while (b - a > 1) {
    const int m = (a + b) / 2;
    if (ps->base[m] <= i) a = m; else b = m;
  }
  i -= ps->base[a];
  r.batch = 0;
  for (int s = a * ((p.nseq + kPromptPlanThreads - 1) / kPromptPlanThreads);; ++s) {
    r.len = prompt_seq(p, s, &r.begin, false);
    const int nb = (r.len + rows - 1) / rows;
    if (i < nb) {
      r.row0 = (nb - 1 - i) * rows;
      return r;
    }
    i -= nb;
  }
}

// Upper bound of the number of query blocks per head, known on the host.
inline int prompt_blocks(const PromptParams& p, int rows) {
  return p.cu ? p.s / rows + (p.nseq < p.s ? p.nseq : p.s) : (p.s + rows - 1) / rows * p.b;
}

}  // namespace mla
