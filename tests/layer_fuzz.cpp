// layer_fuzz.cpp -- the layer products' argument checks and plans (plain C++)
// under the host sanitizers: random and extreme arguments.  Whatever passes the
// checks must plan without overflow, into workspaces and grids that hold
// together.  Prints the number of accepted plans.
#include <cstdint>
#include <cstdio>
#include <random>

#include "plan_layer.h"

using namespace dg;

static std::mt19937_64 rng(12345);

static int64_t dim() {
  static const int64_t edge[] = {0, 1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257,
                                 4096, (1 << 16) + 1, (1 << 22) - 8, (1LL << 31) - 1024,
                                 (1LL << 31) - 1023, 1 << 20, (1LL << 31) - 1,
                                 1LL << 31, INT64_MAX, -1};
  const uint64_t r = rng();
  if (r % 3 == 0) return edge[(r >> 8) % (sizeof(edge) / sizeof(edge[0]))];
  return (int64_t)((r >> 8) % (1ull << (1 + (r >> 40) % 24)));
}

static const void* ptr() {
  static const uintptr_t at[] = {0, 1, 2, 4, 16, 18, 256, 4096};
  return (const void*)at[rng() % 8];
}

static int64_t ld(int64_t cols) {
  const uint64_t r = rng();
  if (r % 4 == 0) return dim();
  return cols < (1LL << 40) && cols >= 0 ? cols + (int64_t)(r >> 8) % 17 : cols;
}

#define REQUIRE(x)                                            \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      return 1;                                               \
    }                                                         \
  } while (0)

int main() {
  long planned = 0;
  for (int it = 0; it < 400000; ++it) {
    const int64_t M = dim(), N = dim(), K = dim();
    const int64_t cus = 1 + (int64_t)(rng() % 512);
    dense_gemm_groups g = {ptr(), rng() % 4 == 0 ? dim() : (int64_t)(rng() % 300), 0};
    const bool grouped = rng() % 2 != 0;
    bool done;
    if (rng() % 2) {
      const int op = (int)(rng() % 5) - (int)(rng() % 8 == 0);
      const int layout = op == DENSE_GEMM_NN_BF16 || op == DENSE_GEMM_NN_F16 ? NN : NT;
      const int64_t lda = ld(K), ldb = ld(layout == NT ? K : N), ldd = ld(N);
      g.stride = rng() % 8 == 0 ? dim() : (ldb > 0 && ldb < (1LL << 31) ? 1024 * ldb : 0);
      dense_gemm_epilogue e = {ptr(), dim(), ptr(), ld(N), (void*)ptr(), ld(N), (int)(rng() % 7) - 1,
                               (int)(rng() % 3)};
      if (rng() % 2) e = {nullptr, 0, nullptr, 0, nullptr, 0, (int)(rng() % 5), 0};
      const void *A = ptr(), *B = ptr(), *D = ptr();
      if (layer_validate(op, M, N, K, A, lda, B, ldb, D, ldd, rng() % 8 ? &e : nullptr,
                         grouped ? &g : nullptr, &done) != DENSE_GEMM_OK || done)
        continue;
      if (grouped) {
        GroupedPlan p;
        if (grouped_plan(layout, M, N, K, A, lda, B, ldb, g, cus, &p) != DENSE_GEMM_OK) continue;
        REQUIRE(p.grid > 0 && p.grid < (1LL << 31));
        REQUIRE(p.tiles_n * p.tile_n >= N && (p.tiles_n - 1) * p.tile_n < N);
        // a launch of one workgroup per tile has room for every way to
        // divide the rows: for one group, and for as many as there can be
        const int64_t active = g.count < M ? g.count : M;
        if (p.small)
          REQUIRE(p.grid >= ((M + p.tile_m - 1) / p.tile_m) * p.tiles_n && p.grid >= active * p.tiles_n);
        REQUIRE((p.a_bytes == 0) == p.a_direct || K == 0);
        REQUIRE(p.a_bytes % 256 == 0 && p.b_bytes % 256 == 0);
      } else {
        CallPlan p;
        if (layer_plan(layout, M, N, K, A, lda, B, ldb, cus, &p) != DENSE_GEMM_OK) continue;
        const int64_t* q = p.plan;
        REQUIRE(q[0] * q[3] >= M && q[1] * q[4] >= N && q[8] >= 1);
        REQUIRE(p.full_tasks + p.split_tiles == q[3] * q[4] || p.small());
        if (!p.small()) {
          REQUIRE(q[8] == 1 || q[8] * q[9] * BK >= K);
          const size_t parts = q[8] > 1 ? (size_t)(q[8] * p.split_tiles) : 0;
          REQUIRE(p.split_bytes >= parts * q[0] * q[1] * sizeof(float));
        }
      }
    } else {
      const int64_t lda = ld(M), ldb = ld(N), ldd = ld(N);
      const void *A = ptr(), *B = ptr(), *D = ptr(), *sums = ptr();
      g.stride = rng() % 8 == 0 ? dim() : (M < (1 << 24) && ldd > 0 && ldd < (1 << 24) ? M * ldd : dim());
      if (tn_validate((int)(rng() % 3) - (int)(rng() % 8 == 0), M, N, K, A, lda, B, ldb, D, ldd, sums,
                      grouped ? &g : nullptr, &done) != DENSE_GEMM_OK || done)
        continue;
      TnPlan p;
      if (tn_plan(M, N, K, A, lda, B, ldb, sums != nullptr, grouped ? &g : nullptr, cus, &p) !=
          DENSE_GEMM_OK)
        continue;
      const int64_t tasks = p.tiles_m * p.tiles_n * p.groups;
      REQUIRE(p.tile * p.tiles_m >= M && p.tile * p.tiles_n >= N);
      REQUIRE(p.full_tasks + p.split_tiles == tasks && p.splits >= 1);
      REQUIRE(tasks <= kLayerMaxTiles);
      // (a workgroup's next task is looked for one round past the last)
      REQUIRE(p.full_tasks + p.splits * p.split_tiles + 2 * cus < (1LL << 31));
      REQUIRE(grouped || p.splits == 1 || p.splits * p.steps * BK >= K);
      REQUIRE(!grouped || p.splits == 1 || p.full_tasks == 0);
      const size_t all = (size_t)(p.full_tasks + p.splits * p.split_tiles);
      // (without: whole tiles write them)
      REQUIRE(sums == nullptr || p.sums_bytes == all * 2 * p.tile * sizeof(float) ||
              (p.sums_bytes == 0 && p.splits == 1));
      REQUIRE(p.splits == 1 || p.split_bytes >= (size_t)(p.splits * p.split_tiles) * p.tile * p.tile * 4);
    }
    ++planned;
  }
  std::printf("planned %ld\n", planned);
  return planned > 1000 ? 0 : 1;
}
