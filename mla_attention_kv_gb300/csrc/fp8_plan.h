// fp8_plan.h -- which kernel takes a call of the e4m3 linear layer, and how the
// kernel for few rows splits it.  Host code.
#pragma once
#include "fp8.h"

namespace mla {

struct NwPlan {
  int tokens, split;
  long long cost;
};

// CTAs of a cluster that share a tile's K blocks: as many as leave a block
// each and two CTAs per SM in all, up to 8, or 4 for tiles of 64 tokens, whose
// sums are larger (64 x 7168 -> 2112 on tiles of 64: 10.0 us on 4, 11.3 on 8;
// one row 8.2 on 4, 7.4 on 8).  Cost: the blocks that the busiest SM takes in
// turn, in units of about 0.15 us: one for a block of up to 32 tokens, two for 64.
// (Splits are powers of two, so the last doubling may leave some SMs with two
// CTAs and others with one: 64 x 16384 -> 7168 has 224 on 152 SMs.)
inline NwPlan plan_for(const Fp8LinearParams& p, int num_sms, int tokens) {
  const int most = tokens == 64 ? 4 : 8;
  const long long blocks = (p.K + kFp8Block - 1) / kFp8Block, tiles = (long long)((p.N + 127) / 128) * ((p.T + tokens - 1) / tokens);
  int split = 1;
  while (split < most && 2 * split <= blocks && tiles * split * 2 <= 2 * num_sms) split *= 2;
  return {tokens, split, (tiles * split + num_sms - 1) / num_sms * ((blocks + split - 1) / split) * (tokens == 64 ? 2 : 1)};
}

// Tiles of 64 tokens, where there are more than 32, unless tiles of 32 find
// SMs without work: 64 x 7168 -> 2112 9.4 us on 32, 10.0 on 64 (cost 14, 28); 64
// x 2048 -> 2048 6.8 and 6.4 (4, 8); 64 x 16384 -> 7168 33.8 and 26.4 (128, 128).
inline NwPlan make_plan(const Fp8LinearParams& p, int num_sms) {
  const NwPlan a = plan_for(p, num_sms, p.T <= 16 ? 16 : 32);
  if (p.T <= 32) return a;
  const NwPlan b = plan_for(p, num_sms, 64);
  return a.cost + 8 <= b.cost ? a : b;
}

// A block of the wide kernel's tile takes three units.  1 x 1536 -> 24576: 9.5
// us on the narrow kernel, 12.6 there (cost 24 and 36); 256 x 7168 -> 2112: 14.2 and 29.4 (56,
// 168); 128 x 1536 -> 24576: 19.6 and 12.4 (72, 36); 256 x 16384 -> 7168: 72 and
// 63 (512, 384); 512 x 2048 -> 576: 7.8 and 10.1 (16, 48).
inline bool fp8_narrow_is_faster(const Fp8LinearParams& p, int num_sms) {
  const long long tiles = (long long)((p.T + 127) / 128) * ((p.N + 255) / 256), blocks = (p.K + kFp8Block - 1) / kFp8Block;
  return make_plan(p, num_sms).cost <= (tiles + num_sms - 1) / num_sms * blocks * 3;
}

}  // namespace mla
