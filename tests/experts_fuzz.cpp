// experts_fuzz.cpp -- the checks and plans of the int8 products and of the
// operators around an expert layer's products (plain C++) under the host
// sanitizers: random and extreme arguments.  Whatever passes the checks must plan
// without overflow, into workspaces and grids that hold together.  Prints the
// number of accepted plans.
#include <cstdint>
#include <cstdio>
#include <random>

#include "plan_experts.h"

using namespace dg;

static std::mt19937_64 rng(54321);

static int64_t dim() {
  static const int64_t edge[] = {0, 1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1024,
                                 1025, 4096, (1 << 17) - 1, 1 << 17, (1 << 16) + 1, (1 << 23) - 8,
                                 (1LL << 31) - 1024, (1LL << 31) - 1023, 1 << 20, (1LL << 31) - 1,
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
    bool done;
    switch (rng() % 4) {
      case 0: {
        const int64_t M = dim(), N = dim(), K = dim(), lda = ld(K), ldb = ld(K);
        const int64_t cus = 1 + (int64_t)(rng() % 512);
        dense_gemm_groups g = {ptr(), rng() % 4 == 0 ? dim() : (int64_t)(rng() % 300),
                               rng() % 8 == 0 ? dim() : (ldb > 0 && ldb < (1LL << 31) ? 1024 * ldb : 0)};
        const bool grouped = rng() % 2 != 0;
        dense_gemm_epilogue e = {ptr(), dim(), ptr(), ld(N), (void*)ptr(), ld(N), (int)(rng() % 7) - 1,
                                 (int)(rng() % 3)};
        if (rng() % 2) e = {nullptr, 0, nullptr, 0, nullptr, 0, (int)(rng() % 5), 0};
        const void *A = ptr(), *B = ptr();
        if (i8_validate((int)(rng() % 4) - 1, M, N, K, A, lda, ptr(), B, ldb, ptr(), ptr(), ld(N), &e,
                        grouped ? &g : nullptr, dim(), &done) != DENSE_GEMM_OK || done)
          break;
        REQUIRE(K <= I8_MOST_K && M > 0 && N > 0);
        if (grouped) {
          GroupedPlan p;
          if (i8_grouped_plan(M, N, K, A, lda, B, ldb, g, cus, &p) != DENSE_GEMM_OK) break;
          REQUIRE(p.grid > 0 && p.grid < kMaxDim && p.tiles_n * p.tile_n >= N);
          REQUIRE(p.a_direct || p.a_bytes >= (size_t)M * K);
          REQUIRE(p.b_direct || p.b_bytes >= (size_t)N * K);
          REQUIRE(!p.a_direct || K == 0 || (((uintptr_t)A | lda) & 3) == 0);
          REQUIRE(p.small || !p.b_direct || K % 4 == 0);
        } else {
          CallPlan p;
          if (i8_plan(M, N, K, A, lda, B, ldb, cus, &p) != DENSE_GEMM_OK) break;
          REQUIRE(p.plan[3] * p.plan[0] >= M && p.plan[4] * p.plan[1] >= N);
          REQUIRE(p.full_tasks + p.split_tiles == p.plan[3] * p.plan[4]);
          REQUIRE(p.a_direct || p.a_bytes >= (size_t)M * K);
          REQUIRE(p.b_direct || p.b_bytes >= (size_t)N * K);
          REQUIRE(p.plan[8] == 1 || p.split_bytes >= (size_t)(p.plan[8] * p.split_tiles) * p.plan[0] * p.plan[1] * 4);
          REQUIRE(p.plan[8] * p.plan[9] * BK * 2 >= K);
        }
        ++planned;
        break;
      }
      case 1: {
        const int64_t T = dim(), n_e = rng() % 4 ? 1 + (int64_t)(rng() % 1100) : dim();
        const int64_t k = rng() % 4 ? 1 + (int64_t)(rng() % 70) : dim();
        dense_gemm_routing r = {ptr(), (int)(rng() % 4) - 1, (int)(rng() % 3), 1.0f, (int)(rng() % 70),
                                (int)(rng() % 8), (int)(rng() % 4)};
        if (route_validate((int)(rng() % 5) - 1, T, n_e, k, ptr(), ld(n_e), &r, ptr(), ptr(), ptr(), ptr(),
                           ptr()) != DENSE_GEMM_OK)
          break;
        const RoutePlan p = route_plan(T, n_e);
        REQUIRE(n_e <= ROUTE_MOST_EXPERTS && k <= ROUTE_MOST_K && T * k < kMaxDim);
        REQUIRE(p.blocks >= 1 && p.chunks * 64 < 65536 && p.blocks * p.chunks * 64 >= T);
        REQUIRE((p.blocks - 1) * p.chunks * 64 < T || T == 0);
        REQUIRE(p.blocks == 1 || p.bytes >= (size_t)(p.blocks * ((n_e + 1) / 2) * 4));
        REQUIRE(r.groups * (n_e / r.groups) == n_e && k <= n_e / r.groups * r.top_groups);
        ++planned;
        break;
      }
      case 2: {
        const int64_t R = dim(), K = dim(), x_rows = dim();
        const void *X = ptr(), *rows = ptr();
        if (quantize_validate((int)(rng() % 4) - 1, R, K, X, ld(K), x_rows, rows, ptr(), ld(K), ptr(), &done) !=
                DENSE_GEMM_OK || done)
          break;
        const int lanes = row_lanes(R, K, 256);
        REQUIRE(lanes == 16 || lanes == 64 || lanes == 256 || lanes == 1024);
        REQUIRE(rows != nullptr || R <= x_rows);
        REQUIRE(K == 0 || x_rows == 0 || X != nullptr);
        ++planned;
        break;
      }
      default: {
        const int64_t T = dim(), N = dim(), k = rng() % 4 ? (int64_t)(rng() % 70) : dim(), rows = dim();
        const void *a = ptr(), *b = ptr();
        if (rng() % 2) {
          if (combine_validate((int)(rng() % 4) - 1, T, N, k, a, ld(N), rows, ptr(), ptr(), b, ld(N), ptr(),
                               ld(N), &done) != DENSE_GEMM_OK || done)
            break;
        } else if (combine_grad_validate((int)(rng() % 4) - 1, T, N, k, a, ld(N), b, ld(N), rows, ptr(), ptr(),
                                         ptr(), ld(N), ptr(), &done) != DENSE_GEMM_OK || done) {
          break;
        }
        REQUIRE(T > 0 && N > 0 && k >= 1 && k <= ROUTE_MOST_K && T * k < kMaxDim);
        ++planned;
      }
    }
  }
  std::printf("planned %ld\n", planned);
  return planned > 5000 ? 0 : 1;
}
