// Host program that answers which kernel an mx4_linear call takes: for every line
// "M N K groups has_a_scale" of standard input it prints "kernel rows max_tiles bytes", or
// "unsupported".
#include <cstdio>

#include "mx4_plan.h"

using namespace moe_mx;

int main() {
  long long M, N, K;
  int groups, scaled;
  while (std::scanf("%lld %lld %lld %d %d", &M, &N, &K, &groups, &scaled) == 5) {
    mx4_linear_problem_t p = {};
    p.M = M;
    p.N = N;
    p.K = K;
    p.groups = groups;
    const mx_linear_problem_t q = as_mxfp8(p);
    if (!linear_sizes_ok(q) || !linear_supported(q) || M == 0) {
      std::puts("unsupported");
      continue;
    }
    const Mx4Plan f = mx4_plan(p, scaled != 0);
    const char* name = f.kind == Fc4::kFew ? "few" : f.kind == Fc4::kWiden ? "widen" : f.ksplit > 1 ? "ranges" : "tile";
    std::printf("%s %d %d %zu\n", name, f.rows, f.max_tiles, f.total);
  }
  return 0;
}
