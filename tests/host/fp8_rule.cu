// fp8_rule.cu -- which kernel takes a call of the e4m3 linear layer (fp8_plan.h).
// With arguments "SMs T K N T K N ...": prints "narrow" or "wide" for each size.
// Without: the choices stay within what a launch can have.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "../../mla_attention_kv_gb300/csrc/fp8_plan.h"

using namespace mla;

static Fp8LinearParams size(int T, int K, int N) {
  Fp8LinearParams p = {};
  p.T = T; p.K = K; p.N = N;
  return p;
}

int main(int argc, char** argv) {
  if (argc > 1) {
    for (int i = 2; i + 2 < argc; i += 3)
      printf("%s\n", fp8_narrow_is_faster(size(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2])), atoi(argv[1])) ? "narrow" : "wide");
    return 0;
  }
  std::mt19937_64 g(1);
  auto log_to = [&](double most) { return std::exp(std::uniform_real_distribution<double>(0, std::log(most))(g)); };
  int failed = 0, checks = 0;
  for (int it = 0; it < 400000; ++it) {
    const int T = (int)log_to(2147418112.0), K = 16 * (int)log_to(134213632.0), N = 8 * (int)log_to(1048560.0);
    if ((double)T * K > 1.1e12 || (double)K * N > 1.1e12 || (double)T * N > 1.1e12) continue;  // (operands and results of a terabyte)
    const int sms = it % 3 == 0 ? 1 + (int)(g() % 300) : 152;
    const Fp8LinearParams p = size(T, K, N);
    const NwPlan a = make_plan(p, sms);
    const long long blocks = (K + 127) / 128, y = (N + 127) / 128, z = ((long long)T + a.tokens - 1) / a.tokens;
    ++checks;
    bool ok = (a.tokens == 16 || a.tokens == 32 || a.tokens == 64) && (a.split == 1 || a.split == 2 || a.split == 4 || a.split == 8) &&
              a.split <= blocks && a.cost > 0;
    // the narrow kernel's grid is split x weight tiles x token tiles
    if (fp8_narrow_is_faster(p, sms)) ok = ok && y <= 65535 && z <= 65535;
    if (!ok && ++failed < 20) printf("failed T %d K %d N %d SMs %d: tokens %d split %d\n", T, K, N, sms, a.tokens, a.split);
  }
  printf("%d checks, %d failed checks\n", checks, failed);
  return failed != 0;
}
