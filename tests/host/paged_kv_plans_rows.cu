// paged_kv_plans_rows.cu -- the checks of paged_kv_plans.cu for the items of
// every kernel form: 4 rows (int8, up to 4 rows), 8 (up to 8) and 16.
#define main paged_kv_plans_main
#include "paged_kv_plans.cu"
#undef main

int main() {
  std::mt19937 g(2);
  auto r = [&](int a, int b) { return a + (int)(g() % (unsigned)(b - a + 1)); };
  // a decode batch over an int8 cache, one row per head; one sequence; rows that fill the last item partly
  run(std::vector<int>(16, 1), {1024, 4096, 2000, 1500, 3333, 1025, 4000, 2048, 1100, 1234, 2345, 3456, 4095, 1999, 2777, 3000}, 1, 128,
      kKvRowsSplit, 1216, 256, 0, true);
  run({1}, {777}, 1, 16, kKvRowsSplit, 1216, 256, 0, true);
  run({3, 0, 1, 7}, {9000, 5, 1, 40}, 1, 5, kKvRowsSplit, 1216, 256, 2, false);
  run({1, 1, 1}, {50000, 0, 300}, 20, 2, kKvRowsSplit, 1216, 256, 0, true);
  const int Rs[] = {kKvRowsSplit, kKvRowsT, kKvRows};
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
    run(n, L, Gs[r(0, 6)], KHs[r(0, 3)], Rs[it % 3], r(0, 3) == 0 ? r(1, 9) : r(600, 1300), 256, r(0, 5), uniform);
  }
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
