// Prints plan_matmul's choice for the device and sizes given: nine cluster counts (pairs, then clusters of
// 1 .. 8), then m n kb per line of standard input.
#include <cstdio>

#include "train_plan.h"

int main() {
  demo::Clusters c;
  for (int& n : c.of)
    if (std::scanf("%d", &n) != 1) return 1;
  long long m, n;
  int kb;
  while (std::scanf("%lld %lld %d", &m, &n, &kb) == 3) {
    const demo::MatmulPlan p = demo::plan_matmul(c, m, n, kb);
    std::printf("%d %d %d %d %d %d %d %u\n", p.group, p.bn, p.split, p.stages, p.rows_a, p.rows_b, p.chain, p.grid);
  }
  return 0;
}
