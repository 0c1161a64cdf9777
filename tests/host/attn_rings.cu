// attn_rings.cu -- host model of how a copying role of the attention kernels
// leaves its ring of slots (attn_tc.cuh, ring_uses) when a wait runs out at
// any point: no final wait may return at once while the slot's last fill has
// not been released.  A barrier is its number of completed phases; a wait for
// parity P returns when the phase under way does not have parity P.
#include <cstdio>
#include <random>
#include <vector>

#include "../../mla_attention_kv_gb300/csrc/attn_tc.cuh"

using namespace mla;

static int failed = 0, checks = 0;
#define CHECK(...)                                                            \
  do {                                                                        \
    ++checks;                                                                 \
    if (!(__VA_ARGS__) && ++failed < 20) printf("failed %s line %d\n", #__VA_ARGS__, __LINE__); \
  } while (0)

static bool passes(uint32_t phases, uint32_t parity) { return (phases & 1) != parity; }

int main() {
  std::mt19937 g(3);
  int whole_rounds_wrong = 0;
  for (int it = 0; it < 20000; ++it) {
    const uint32_t slots = 2 + g() % 3, rounds = 1 + g() % 6;
    std::vector<uint32_t> empty(slots, 0), filled(slots, 0);
    // the role fills slots in turn, the reader releases them in turn some way behind, and stops somewhere
    uint32_t fills = 0, released = 0, u = 0;
    const uint32_t stop = g() % (slots * rounds + 1);  // releases that come before the wait's limit
    bool ok = true;
    for (; u < rounds && ok; ++u)
      for (uint32_t s = 0; s < slots; ++s) {
        while (!passes(empty[s], (u & 1) ^ 1) && released < stop && released < fills) ++empty[released++ % slots];
        if (!passes(empty[s], (u & 1) ^ 1)) {
          ok = false;
          break;
        }
        ++filled[s];
        ++fills;
      }
    for (uint32_t s = 0; s < slots; ++s) {
      const uint32_t n = ring_uses(fills, slots, s);
      CHECK(n == filled[s]);
      if (n == 0) continue;
      CHECK(passes(empty[s], (n - 1) & 1) == (empty[s] == n));
      whole_rounds_wrong += !ok && passes(empty[s], (u - 1) & 1) && empty[s] != n;
    }
  }
  CHECK(whole_rounds_wrong > 0);  // (the model does tell the two apart)
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
