// Host program that answers which kernel an mx_linear call takes: for every line
// "M N K groups act w_fmt has_a_scale" (numbers) of standard input it prints
// "kernel rows ksplit workgroups max_tiles bytes", workgroups being the grid of the
// few-row kernel (one per item) and 0 for the persistent ones, or "unsupported".
#include <cstdio>

#include "linear_plan.h"

using namespace moe_mx;

int main() {
  long long M, N, K;
  int groups, act, fmt, scaled;
  while (std::scanf("%lld %lld %lld %d %d %d %d", &M, &N, &K, &groups, &act, &fmt, &scaled) == 7) {
    mx_linear_problem_t p = {};
    p.M = M;
    p.N = N;
    p.K = K;
    p.groups = groups;
    p.act = (moe_act_t)act;
    p.w_fmt = (mx_elem_t)fmt;
    if (!linear_sizes_ok(p) || !linear_supported(p) || M == 0) {
      std::puts("unsupported");
      continue;
    }
    const LinearPlan f = linear_plan(p, scaled != 0);
    const char* name = f.kind == Fc::kFew ? "few" : f.kind == Fc::kRows ? "rows" : f.kind == Fc::kMid ? "mid"
                       : f.kind == Fc::kTiled ? "tiled" : f.kind == Fc::kWide ? "wide" : "none";
    const long long tiles = groups > 0 ? f.max_tiles : (M + f.rows - 1) / f.rows;
    const long long wgs = f.kind == Fc::kFew ? tiles * ((N + kFewCols - 1) / kFewCols) : 0;
    std::printf("%s %d %d %lld %lld %zu\n", name, f.rows, f.ksplit, wgs, tiles, f.total);
  }
  return 0;
}
