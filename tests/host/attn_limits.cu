// attn_limits.cu -- host check of the paged attention's plan (paged_plan.cuh)
// at the longest sequences that 32-bit lengths name.  A table may repeat its
// blocks, so such a length needs neither a large cache nor a large table.
#include <cstdio>

#include "../../mla_attention_kv_gb300/csrc/paged_plan.cuh"

using namespace mla;

static int failed = 0, checks = 0;
#define CHECK(...)                                                            \
  do {                                                                        \
    ++checks;                                                                 \
    if (!(__VA_ARGS__) && ++failed < 20) printf("failed %s line %d\n", #__VA_ARGS__, __LINE__); \
  } while (0)

int main() {
  const int lens[] = {0x7fffffff, 0x7fffffff - 62, 0x7fffffff - 126, 0x7fffff01, 0x7fffff00, 0x7ffffeff, 1 << 30};
  const int heads[] = {1, 16, 128}, rows[] = {16, 32, 128};
  for (int L : lens)
    for (int H : heads)
      for (int R : rows)
        for (int n : {1, 2, 300}) {
          const int cu[] = {0, n};
          PagedParams p = {};
          p.cu_q = cu; p.kv_lens = &L; p.nseq = 1; p.T = n; p.heads = H; p.page = 65536; p.table_stride = 32768; p.workers = 76;
          const Seq q = plan_seq(p, 0, R, false);
          CHECK(q.L == (L < kMaxKeys ? L : kMaxKeys));
          for (int j : {0, q.items - 1}) {
            const int keys = q.keys_of_item(j, R, H);
            CHECK(keys > 0 && keys <= q.L);
            for (long long tile : {32, 64, 128}) {
              const long long tiles = (keys + tile - 1) / tile;
              CHECK((int)((keys + (int)(tile - 1)) / (int)tile) == tiles);
              CHECK((tiles + 1) * tile - 1 <= 0x7fffffffLL);  // the last key number of the tile behind the last one
            }
          }
          CHECK(q.first > 0 && q.last >= q.first && q.cum(q.items) >= (long long)q.items * q.first);
        }
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
