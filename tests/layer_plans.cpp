// layer_plans.cpp -- prints the plans of the layer products, one line for each
// line read: contiguous, 256-byte aligned operands on `cus` CUs.
//   layer LAYOUT M N K        tile rows, tile columns (16: the small-output
//                             kernel), tiles, parts of K, tiles in parts,
//                             operands copied
//   grouped LAYOUT M N K G    the same, tiles and parts as the host knows them
//   tn M N K G SUMS           the same, then the bytes of partial column sums;
//                             G = 0: no groups
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "plan_layer.h"

using namespace dg;

static void out(int64_t tm, int64_t tn, int64_t tiles, int64_t parts, int64_t split, bool a, bool b) {
  std::printf("%lld %lld %lld %lld %lld %d", (long long)tm, (long long)tn, (long long)tiles,
              (long long)parts, (long long)split, (int)!a + (int)!b);
}

int main(int argc, char** argv) {
  const int64_t cus = argc > 1 ? std::atoll(argv[1]) : 256;
  const void* p = (const void*)256;
  char kind[16];
  while (std::scanf("%15s", kind) == 1) {
    long long x[5] = {};
    const int n = kind[0] == 'l' ? 4 : 5;
    for (int i = 0; i < n; ++i)
      if (std::scanf("%lld", &x[i]) != 1) return 1;
    if (kind[0] == 'l') {
      CallPlan c;
      const int64_t N = x[2], K = x[3];
      if (layer_plan((int)x[0], x[1], N, K, p, K, p, x[0] == NT ? K : N, cus, &c) != DENSE_GEMM_OK) return 1;
      out(c.plan[0], c.plan[1], c.plan[3] * c.plan[4], c.plan[8], c.split_tiles, c.a_direct, c.b_direct);
    } else if (kind[0] == 'g') {
      GroupedPlan g;
      const int64_t N = x[2], K = x[3];
      const dense_gemm_groups gr = {p, x[4], N * K};
      if (grouped_plan((int)x[0], x[1], N, K, p, K, p, x[0] == NT ? K : N, gr, cus, &g) != DENSE_GEMM_OK)
        return 1;
      out(g.tile_m, g.tile_n, g.grid, 1, 0, g.a_direct, g.b_direct);
    } else {
      TnPlan t;
      const int64_t M = x[0], N = x[1];
      const dense_gemm_groups gr = {p, x[3], M * N};
      if (tn_plan(M, N, x[2], p, M, p, N, x[4] != 0, x[3] > 0 ? &gr : nullptr, cus, &t) != DENSE_GEMM_OK)
        return 1;
      out(t.tile, t.tile, t.tiles_m * t.tiles_n * t.groups, t.splits, t.split_tiles, t.a_direct, t.b_direct);
      std::printf(" %zu", t.sums_bytes);
    }
    std::printf("\n");
  }
  return 0;
}
