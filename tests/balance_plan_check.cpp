// Host program that answers how moe_balance and its gradient are launched: for every line "T E S"
// of standard input it prints "chunks rows workgroups_of_the_second_launch workspace", then "rows
// workgroups" of the gradient without and with 16-byte pieces, or "unsupported".
#include <cstdio>

#include "balance_plan.h"

using namespace moe_mx;

int main() {
  int T, E, S;
  while (std::scanf("%d %d %d", &T, &E, &S) == 3) {
    if (!balance_sizes_valid(T, E, 1, S) || !balance_sizes_supported(T, E, 1, S)) {
      std::puts("unsupported");
      continue;
    }
    const BalancePlan f = balance_plan(T, E, S);
    std::printf("%d %d %lld %zu", f.chunks, f.rows, (long long)S * f.blocks, f.total);
    for (int vec = 0; vec < 2; ++vec) {
      if (vec && E % 4) {
        std::printf(" 0 0");
        continue;
      }
      for_row_shape<false>(vec, E, [&](auto, auto L, auto) {
        constexpr int G = kThreadsB / L.value;
        std::printf(" %d %lld", G * balance_grad_rows(T, G), (long long)balance_grad_blocks(T, G));
      });
    }
    std::puts("");
  }
  return 0;
}
