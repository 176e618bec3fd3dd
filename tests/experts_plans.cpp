// experts_plans.cpp -- prints the plans of the int8 products, one line for each
// line read: contiguous, 256-byte aligned operands on `cus` CUs.
//   i8 M N K           tile rows, tile columns (16: the small-output kernel),
//                      tiles, parts of K, tiles in parts, operands copied
//   grouped M N K G    the same, tiles and parts as the host knows them
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "plan_experts.h"

using namespace dg;

int main(int argc, char** argv) {
  const int64_t cus = argc > 1 ? std::atoll(argv[1]) : 256;
  const void* p = (const void*)256;
  char kind[16];
  while (std::scanf("%15s", kind) == 1) {
    long long x[4] = {};
    const int n = kind[0] == 'i' ? 3 : 4;
    for (int i = 0; i < n; ++i)
      if (std::scanf("%lld", &x[i]) != 1) return 1;
    const int64_t M = x[0], N = x[1], K = x[2];
    if (kind[0] == 'i') {
      CallPlan c;
      if (i8_plan(M, N, K, p, K, p, K, cus, &c) != DENSE_GEMM_OK) return 1;
      std::printf("%lld %lld %lld %lld %lld %d\n", (long long)c.plan[0], (long long)c.plan[1],
                  (long long)(c.plan[3] * c.plan[4]), (long long)c.plan[8], (long long)c.split_tiles,
                  (int)!c.a_direct + (int)!c.b_direct);
    } else {
      GroupedPlan g;
      const dense_gemm_groups gr = {p, x[3], N * K};
      if (i8_grouped_plan(M, N, K, p, K, p, K, gr, cus, &g) != DENSE_GEMM_OK) return 1;
      std::printf("%d %d %lld 1 0 %d\n", g.tile_m, g.tile_n, (long long)g.grid,
                  (int)!g.a_direct + (int)!g.b_direct);
    }
  }
  return 0;
}
