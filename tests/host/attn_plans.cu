// attn_plans.cu -- host check of the paged attention's work split
// (paged_plan.cuh): the pieces that the workers take cover every key tile of
// every item once, partial results have a slot of their own, and the records
// that the joining kernel works from (rows, last worker) fit the pieces.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

#include "../../mla_attention_kv_gb300/csrc/paged_plan.cuh"

using namespace mla;

static int failed = 0, checks = 0;
#define CHECK(...)                                                             \
  do {                                                                       \
    ++checks;                                                                \
    if (!(__VA_ARGS__)) {                                                             \
      if (++failed < 20) printf("failed %s line %d\n", #__VA_ARGS__, __LINE__);        \
    }                                                                        \
  } while (0)

static long long host_total(const PagedParams& p, PlanShared* ps, int R, int nt) {
  const int strip = (p.nseq + nt - 1) / nt;
  long long at = 0;
  for (int t = 0; t < nt; ++t) {
    ps->base[t] = at;
    for (int i = 0; i < strip; ++i)
      if (t * strip + i < p.nseq) {
        const Seq q = plan_seq(p, t * strip + i, R, false);
        at += q.cum(q.items);
      }
  }
  ps->base[nt] = at;
  ps->threads = nt;
  return at;
}

struct Piece { int t0, t1, worker, slot; bool whole; };

static void run(const std::vector<int>& n, const std::vector<int>& L, int H, int R, int W, int nt, int lead, bool uniform) {
  std::vector<int> cu = {lead}, lens = L;
  for (int x : n) cu.push_back(cu.back() + x);
  PagedParams p = {};
  p.cu_q = uniform ? nullptr : cu.data();
  p.kv_lens = lens.data();
  p.nseq = (int)n.size();
  p.T = cu.back() + 3;
  p.n_uniform = uniform ? n[0] : 0;
  p.heads = H;
  p.page = 16;
  p.table_stride = 1 << 20;
  p.workers = W;
  static PlanShared ps;
  const long long total = host_total(p, &ps, R, nt);
  std::map<std::pair<int, int>, std::vector<Piece>> got;
  std::map<int, int> slots;
  if (total > 0) {
    const int We = plan_workers(total, W, R);
    CHECK(We >= 1 && We <= W);
    for (int w = 0; w < We; ++w) {
      const long long x0 = plan_worker_begin(total, w, We), x1 = plan_worker_begin(total, w + 1, We);
      CHECK(x1 > x0);
      PlanCursor c;
      c.seek(p, &ps, R, x0);
      CHECK(c.lo <= x0 && x0 < c.hi);
      for (bool more = true; more && c.lo < x1; more = c.next(p, R)) {
        CHECK(c.s >= 0 && c.s < p.nseq && c.j >= 0 && c.j < c.q.items && c.hi > c.lo);
        const int keys = c.q.keys_of_item(c.j, R, H);
        CHECK(keys >= 0 && keys <= c.q.L);
        const int tiles = (keys + kKeyTile - 1) / kKeyTile;
        const long long a = x0 > c.lo ? x0 : c.lo, b = x1 < c.hi ? x1 : c.hi;
        Piece pc = {c.tile_at(a, tiles, R), c.tile_at(b, tiles, R), w, -1, c.lo >= x0 && c.hi <= x1};
        CHECK(pc.t0 >= 0 && pc.t0 <= pc.t1 && pc.t1 <= tiles);
        if (!pc.whole) {
          pc.slot = w * 2 + (c.lo < x0 ? 0 : 1);
          CHECK(++slots[pc.slot] == 1);
        }
        got[{c.s, c.j}].push_back(pc);
      }
    }
    // the records that the joining kernel works from
    std::map<std::pair<int, int>, int> joined;
    std::vector<PagedJoin> joins(W, PagedJoin{-1, -1, -1, -1});
    p.joins = joins.data();
    for (int w = 0; w < We; ++w) {
      const long long x0 = plan_worker_begin(total, w, We), x1 = plan_worker_begin(total, w + 1, We);
      PlanCursor c;
      c.seek(p, &ps, R, x0);
      int posted = 0;
      for (bool more = true; more && c.lo < x1; more = c.next(p, R))
        if (c.hi >= x1) {
          plan_post_join(p, c, R, w, x0, x1, total, We);
          ++posted;
          if (joins[w].rows == 0) continue;
          CHECK(++joined[{c.s, c.j}] == 1);
          const auto& ps2 = got[{c.s, c.j}];
          CHECK(joins[w].row == c.q.begin * H + c.j * R);
          CHECK(joins[w].rows == std::min(R, c.q.n * H - c.j * R));
          CHECK(joins[w].last_worker - w + 1 == (int)ps2.size());
          for (size_t i = 0; i < ps2.size(); ++i) {
            CHECK(ps2[i].worker == w + (int)i);
            CHECK(ps2[i].slot == ps2[i].worker * 2 + (i == 0 ? 1 : 0));
          }
        }
      CHECK(posted == 1 && joins[w].rows >= 0);
    }
    for (auto& kv : got) CHECK((kv.second.size() > 1) == (joined.count(kv.first) == 1));
  }
  for (int s = 0; s < p.nseq; ++s) {
    const Seq q = plan_seq(p, s, R, false);
    CHECK(q.begin == (uniform ? s * n[0] : cu[s]) && q.n == n[s] && q.L == L[s]);
    CHECK(q.items == ((long long)n[s] * H + R - 1) / R);
    for (int j = 0; j < q.items; ++j) {
      const auto& pcs = got[{s, j}];
      CHECK(!pcs.empty());
      const int rows_end = std::min((j + 1) * R, n[s] * H), t = (rows_end - 1) / H;
      const int keys = std::max(0, L[s] - n[s] + t + 1);
      CHECK(q.keys_of_item(j, R, H) == keys);
      int at = 0;
      for (const Piece& pc : pcs) {
        CHECK(pc.t0 == at);
        at = pc.t1;
        CHECK(pc.whole == (pcs.size() == 1));
      }
      CHECK(at == (keys + kKeyTile - 1) / kKeyTile);
    }
  }
}

int main() {
  std::mt19937 g(1);
  auto r = [&](int a, int b) { return a + (int)(g() % (unsigned)(b - a + 1)); };
  run({0, 1, 3, 5, 2, 70, 0, 9}, {5, 1, 2, 0, 90, 200, 0, 9}, 5, 32, 152, 256, 2, false);
  for (int H : {5, 16, 40, 128}) for (int R : {16, 32, 128}) run({0, 1, 3, 5, 2, 70, 0, 9}, {5, 1, 2, 0, 90, 200, 0, 9}, H, R, 152, 256, 2, false);
  run({0, 0}, {5, 0}, 16, 16, 152, 256, 0, false);
  run({1}, {0}, 16, 16, 152, 256, 0, true);
  run({1}, {131072}, 128, 128, 76, 256, 0, true);
  run({2048}, {2048}, 128, 128, 76, 384, 0, true);
  run({5000}, {40000}, 128, 128, 76, 256, 0, false);
  for (int it = 0; it < 3000; ++it) {
    const int ns = r(0, 9) == 0 ? r(200, 900) : r(1, 12);
    const bool uniform = r(0, 1);
    const int mode = r(0, 3), un = r(1, 4);
    std::vector<int> n, L;
    for (int i = 0; i < ns; ++i) {
      n.push_back(uniform ? un : (mode == 0 ? 1 : mode == 1 ? r(0, 3) : mode == 2 ? r(0, 40) : r(0, 2) * r(1, 300)));
      L.push_back(r(0, 4) == 0 ? r(0, 3) : r(0, 3) == 0 ? r(0, 40000) : n.back() + r(0, 700));
    }
    const int Hs[] = {1, 3, 5, 8, 16, 20, 64, 128, 200};
    const int Rs[] = {16, 32, 64, 128};
    run(n, L, Hs[r(0, 8)], Rs[r(0, 3)], r(0, 3) == 0 ? r(1, 9) : r(70, 160), r(0, 1) ? 256 : 384, r(0, 5), uniform);
  }
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
