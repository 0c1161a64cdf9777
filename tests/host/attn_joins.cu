// attn_joins.cu -- host check of the records that the paged attention's
// joining kernel works from (paged_plan.cuh) when workers give up: whatever
// an earlier call has left, every record that is read lies within the rows
// and workers of the call that reads it, and one that does not fit is dropped.
#include <cstdio>
#include <random>
#include <vector>

#include "../../mla_attention_kv_gb300/csrc/paged_plan.cuh"

using namespace mla;

static int failed = 0, checks = 0;
#define CHECK(...)                                                            \
  do {                                                                        \
    ++checks;                                                                 \
    if (!(__VA_ARGS__) && ++failed < 20) printf("failed %s line %d\n", #__VA_ARGS__, __LINE__); \
  } while (0)

int main() {
  std::mt19937 g(7);
  auto r = [&](int a, int b) { return a + (int)(g() % (unsigned)(b - a + 1)); };
  static PlanShared ps;
  int cleared = 0, joined = 0;
  for (int it = 0; it < 2000; ++it) {
    const int ns = r(1, 90), H = it & 1 ? 128 : 16, R = it & 2 ? 128 : 32, W = 76, nt = 320;
    std::vector<int> cu = {0}, lens;
    for (int i = 0; i < ns; ++i) {
      cu.push_back(cu.back() + r(0, 3));
      lens.push_back(r(0, 900));
    }
    std::vector<PagedJoin> joins(W, PagedJoin{1 << 24, 128, 303, 0});  // left by a larger call
    PagedParams p = {};
    p.cu_q = cu.data(); p.kv_lens = lens.data(); p.nseq = ns; p.T = cu.back(); p.heads = H; p.page = 16;
    p.table_stride = 1 << 20; p.workers = W; p.joins = joins.data();
    const int strip = (ns + nt - 1) / nt;
    long long total = 0;
    for (int t = 0; t <= nt; ++t) {
      ps.base[t] = total;
      for (int i = 0; t < nt && i < strip; ++i)
        if (t * strip + i < ns) {
          const Seq q = plan_seq(p, t * strip + i, R, false);
          total += q.cum(q.items);
        }
    }
    ps.threads = nt;
    const int We = total > 0 ? plan_workers(total, W, R) : 0;
    for (int w = 0; w < W; ++w) {
      plan_open_join(p, w);  // (every block, before it leaves or waits)
      if (w >= We) continue;
      const long long x0 = plan_worker_begin(total, w, We), x1 = plan_worker_begin(total, w + 1, We);
      PlanCursor c;
      c.seek(p, &ps, R, x0);
      for (bool more = true; more && c.lo < x1; more = c.next(p, R)) {
        if (c.hi >= x1) plan_post_join(p, c, R, w, x0, x1, total, We);
        if (r(0, 1)) break;  // a wait ran out in this item
      }
    }
    for (int w = 0; w < W; ++w) {
      CHECK(joins[w].rows >= 0 && (long long)joins[w].row + joins[w].rows <= (long long)p.T * H);
      if (joins[w].rows == 0) { ++cleared; continue; }
      ++joined;
      CHECK(plan_join_fits(p, joins[w], w, R));
      PagedJoin j = joins[w];
      j.row = p.T * H - j.rows + 1;
      CHECK(!plan_join_fits(p, j, w, R));
      j = joins[w]; j.row = -1;
      CHECK(!plan_join_fits(p, j, w, R));
      j = joins[w]; j.rows = R + 1;
      CHECK(!plan_join_fits(p, j, w, R));
      j = joins[w]; j.last_worker = W;
      CHECK(!plan_join_fits(p, j, w, R));
      j.last_worker = w - 1;
      CHECK(!plan_join_fits(p, j, w, R));
    }
  }
  CHECK(cleared > 1000 && joined > 1000);
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
