// attn_tc.cuh -- helpers shared by the tcgen05 attention kernels: bounded
// waits, TMEM stores of 32 columns, packed fp32 arithmetic, 2^x.
#pragma once
#include "common.cuh"
#include "tc.cuh"

namespace mla {

// A value that is the same in every lane, made known as such to the compiler:
// the operands of tcgen05 and TMA instructions are uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(~0u, v); }

// Bounded mbarrier wait shared by all roles of a CTA; gives up on the time
// budget or when another role has already given up.
// kCluster: some arrivals come from the other CTA of the cluster.
template <bool kCluster = false>
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                        unsigned long long budget, unsigned* status) {
  // (the timer is read only after some tries: reading it costs about as much as a wait usually takes)
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (kCluster ? tc::try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((n & 63) == 0) {
      if (*abort) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > budget) {
        *abort = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}
// The same by polling.  at_wait can overrun a short limit (its try_wait holds
// the thread for a time slice, and 128 of them come before the limit is
// compared); this one keeps any.  The MMA thread's first wait, which always
// lasts some time (for the queries), is made with it: a limit too short for a
// call is then reported by that call.  In every at_wait instead: prompt of
// 8192 1.93 -> 2.12 ms.
template <bool kCluster = false>
__device__ __forceinline__ bool at_wait_poll(uint32_t bar, uint32_t parity, volatile int* abort,
                                             unsigned long long budget, unsigned* status) {
  const uint64_t t0 = globaltimer_ns();
  while (!(kCluster ? tc::test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity))) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > budget) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// at_wait for a whole warp: all lanes get one answer.
__device__ __forceinline__ bool at_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                             unsigned long long budget, unsigned* status) {
  return __all_sync(~0u, at_wait(bar, parity, abort, budget, status));
}

// How often slot i of a ring of `slots` has been filled after `fills` fills in
// turn.  A role that gives up leaves a ring at any place; the barriers of a
// slot filled n > 0 times are then waited on with parity (n - 1) & 1: that of
// its last fill, whose phase is the current one or has just completed.  (A
// parity counted in whole rounds can name the phase before it, which is
// complete, and the wait returns with a copy still in flight.)
__host__ __device__ constexpr uint32_t ring_uses(uint32_t fills, uint32_t slots, uint32_t i) {
  return (fills + slots - 1 - i) / slots;
}

__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x (results below the normal range become 0).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scale `COLS` (a multiple of 16) fp32 TMEM columns of this thread's lane.
template <int COLS>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, float f) {
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    uint32_t v[32];
    tc::ld32(taddr + c, v);
    tc::wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
    tc::st16(taddr + c, v);
    tc::st16(taddr + c + 16, v + 16);
  }
}

}  // namespace mla
