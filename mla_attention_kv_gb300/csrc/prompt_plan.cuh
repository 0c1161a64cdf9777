// prompt_plan.cuh -- which query block of which sequence a CTA of the prompt
// attention works on.
#pragma once
#include "attn.h"
#include "common.cuh"

namespace mla {

struct PromptPlace {
  int batch, begin, len, row0;  // sequence: rows begin .. begin + len of `batch`; first query row in it
};

struct PromptPlanShared {
  int warp_sum[32];
  PromptPlace place;
  int found;
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

// Query block `index` (of `rows` rows) of the call; false past the last
// one.  Blocks of one sequence are taken from its end: causal blocks late in
// a sequence have the most keys and start first.  All threads of the block.
__device__ __forceinline__ bool prompt_place(const PromptParams& p, PromptPlanShared* ps, int index, int rows,
                                             PromptPlace* out, bool report) {
  if (!p.cu) {
    const int per = (p.s + rows - 1) / rows;
    if (index >= per * p.b) return false;
    out->batch = index % p.b;
    out->begin = 0;
    out->len = p.s;
    out->row0 = (per - 1 - index / p.b) * rows;
    return true;
  }
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  if (tid == 0) ps->found = 0;
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < warp; ++w) before += ps->warp_sum[w];
  if (index >= before && index < before + mine) {
    int left = index - before;
    for (int i = 0; i < strip; ++i) {
      const int len = prompt_seq(p, tid * strip + i, &begin, false);
      const int nb = (len + rows - 1) / rows;
      if (left < nb) {
        ps->place = PromptPlace{0, begin, len, (nb - 1 - left) * rows};
        ps->found = 1;
        break;
      }
      left -= nb;
    }
  }
  __syncthreads();
  *out = ps->place;
  return ps->found != 0;
}

// Upper bound of the number of query blocks, known on the host.
inline int prompt_blocks(const PromptParams& p, int rows) {
  return p.cu ? p.s / rows + (p.nseq < p.s ? p.nseq : p.s) : (p.s + rows - 1) / rows * p.b;
}

}  // namespace mla
