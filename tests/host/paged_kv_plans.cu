// paged_kv_plans.cu -- host check of the paged K/V attention's work split
// (paged_kv_plan.cuh): the workers' pieces cover every key tile of every item
// (sequence, KV head, row block) once, partial results have a slot of their
// own, all workers of an item agree on the first and the last of them, and the
// records of the joining kernel fit the pieces.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "../../mla_attention_kv_gb300/csrc/paged_kv_plan.cuh"

using namespace mla;

static int failed = 0, checks = 0;
#define CHECK(...)                                                             \
  do {                                                                         \
    ++checks;                                                                  \
    if (!(__VA_ARGS__)) {                                                      \
      if (++failed < 20) printf("failed %s line %d\n", #__VA_ARGS__, __LINE__); \
    }                                                                          \
  } while (0)

struct Piece { int t0, t1, worker, slot; bool whole; int first, last; };
using Key = std::tuple<int, int, int>;

static void run(const std::vector<int>& n, const std::vector<int>& L, int G, int KH, int R, int W, int nt, int lead, bool uniform) {
  std::vector<int> cu = {lead}, lens = L;
  for (int x : n) cu.push_back(cu.back() + x);
  PagedKvParams p = {};
  p.plan.cu_q = uniform ? nullptr : cu.data();
  p.plan.kv_lens = lens.data();
  p.plan.nseq = (int)n.size();
  p.plan.T = cu.back() + 3;
  p.plan.n_uniform = uniform ? n[0] : 0;
  p.plan.heads = G;
  p.plan.page = 16;
  p.plan.table_stride = 1 << 20;
  p.plan.workers = W;
  p.kv_heads = KH;
  p.item_cost = 1 + (L[0] + KH) % 3;
  static PlanShared ps;
  const int strip = (p.plan.nseq + nt - 1) / nt;
  long long total = 0;
  for (int t = 0; t < nt; ++t) {
    ps.base[t] = total;
    for (int i = 0; i < strip; ++i)
      if (t * strip + i < p.plan.nseq) {
        const Seq q = kv_seq(p, t * strip + i, R, false);
        total += q.cum(q.items) * KH;
      }
  }
  ps.base[nt] = total;
  ps.threads = nt;
  std::map<Key, std::vector<Piece>> got;
  std::map<int, int> slots;
  if (total > 0) {
    const int We = kv_workers(total, W);
    CHECK(We >= 1 && We <= W);
    std::vector<PagedJoin> joins(W, PagedJoin{-1, -1, -1, -1});
    p.plan.joins = joins.data();
    std::map<Key, int> joined;
    for (int w = 0; w < We; ++w) {
      const long long x0 = plan_worker_begin(total, w, We), x1 = plan_worker_begin(total, w + 1, We);
      CHECK(x1 > x0);
      KvCursor c;
      c.seek(p, &ps, R, x0);
      CHECK(c.lo <= x0 && x0 < c.hi);
      for (bool more = true; more && c.lo < x1; more = c.next(p, R)) {
        CHECK(c.s >= 0 && c.s < p.plan.nseq && c.head >= 0 && c.head < KH && c.j >= 0 && c.j < c.q.items && c.hi > c.lo);
        const int keys = c.q.keys_of_item(c.j, R, G), tiles = (keys + kKvTile - 1) / kKvTile;
        const long long a = x0 > c.lo ? x0 : c.lo, b = x1 < c.hi ? x1 : c.hi;
        Piece pc = {c.tile_at(a, tiles), c.tile_at(b, tiles), w, -1, c.lo >= x0 && c.hi <= x1, -1, -1};
        CHECK(pc.t0 >= 0 && pc.t0 <= pc.t1 && pc.t1 <= tiles);
        if (!pc.whole) {
          pc.slot = w * 2 + (c.lo < x0 ? 0 : 1);
          CHECK(++slots[pc.slot] == 1);
        }
        kv_sharers(c, w, x0, x1, total, We, &pc.first, &pc.last);
        got[Key(c.s, c.head, c.j)].push_back(pc);
        if (c.hi >= x1) {
          kv_post_join(p, c, R, w, x0, x1, total, We);
          if (joins[w].rows > 0) {
            CHECK(++joined[Key(c.s, c.head, c.j)] == 1);
            CHECK(joins[w].row == c.q.begin * G + c.j * R && joins[w].pad == c.head);
            CHECK(joins[w].rows == std::min(R, c.q.n * G - c.j * R));
          }
        }
      }
      CHECK(joins[w].rows >= 0);
    }
    std::map<int, int> begun;  // split items that a worker begins
    for (auto& kv : got) {
      const auto& v = kv.second;
      CHECK((v.size() > 1) == (joined.count(kv.first) == 1));
      if (v.size() > 1) CHECK(++begun[v[0].worker] == 1 && joins[v[0].worker].last_worker == v.back().worker);
      for (size_t i = 0; i < v.size(); ++i) {
        CHECK(v[i].first == v[0].worker && v[i].last == v.back().worker && v[i].worker == v[0].worker + (int)i);
        if (v.size() > 1) CHECK(v[i].slot == v[i].worker * 2 + (i == 0 ? 1 : 0));
      }
    }
  }
  size_t items = 0;
  for (int s = 0; s < p.plan.nseq; ++s) {
    const int per = (int)(((long long)n[s] * G + R - 1) / R);
    for (int h = 0; h < KH; ++h)
      for (int j = 0; j < per; ++j, ++items) {
        const auto& v = got[Key(s, h, j)];
        CHECK(!v.empty());
        const int rows_end = std::min((j + 1) * R, n[s] * G), keys = std::max(0, L[s] - n[s] + (rows_end - 1) / G + 1);
        int at = 0;
        for (const Piece& pc : v) {
          CHECK(pc.t0 == at && pc.whole == (v.size() == 1));
          at = pc.t1;
        }
        CHECK(at == (keys + kKvTile - 1) / kKvTile);
      }
  }
  CHECK(items == got.size());
}

int main() {
  std::mt19937 g(1);
  auto r = [&](int a, int b) { return a + (int)(g() % (unsigned)(b - a + 1)); };
  run({0, 0}, {5, 0}, 1, 16, 16, 1216, 256, 0, false);
  run({1}, {0}, 1, 16, 16, 1216, 256, 0, true);
  run({1}, {777}, 1, 16, 16, 1216, 256, 0, true);
  run({1}, {131072}, 1, 128, 8, 1216, 256, 0, true);
  run({300}, {2048}, 4, 8, 16, 1216, 256, 0, true);
  for (int it = 0; it < 1500; ++it) {
    const int ns = r(0, 9) == 0 ? r(200, 600) : r(1, 12);
    const bool uniform = r(0, 1);
    const int mode = r(0, 3), un = r(1, 4);
    std::vector<int> n, L;
    for (int i = 0; i < ns; ++i) {
      n.push_back(uniform ? un : (mode == 0 ? 1 : mode == 1 ? r(0, 3) : mode == 2 ? r(0, 40) : r(0, 2) * r(1, 60)));
      L.push_back(r(0, 4) == 0 ? r(0, 3) : r(0, 9) == 0 ? r(0, 9000) : n.back() + r(0, 700));
    }
    const int Gs[] = {1, 2, 3, 4, 8, 16, 20}, KHs[] = {1, 2, 5, 16};
    run(n, L, Gs[r(0, 6)], KHs[r(0, 3)], r(0, 1) ? 8 : 16, r(0, 3) == 0 ? r(1, 9) : r(600, 1300), r(0, 1) ? 256 : 352, r(0, 5), uniform);
  }
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
