// plan_layer.cpp -- argument checks, launch plans and workspace sizes of a
// layer's products (plan_layer.h).  Plain C++ with no device code, so it also
// builds with the host sanitizers.
#include "plan_layer.h"

namespace dg {

namespace {

constexpr size_t kMaxBytes = (size_t)1 << 62;

// a * b * 2 bytes, rounded up to 256; false past kMaxBytes
bool matrix_bytes(int64_t a, int64_t b, size_t* out) {
  size_t n;
  if (__builtin_mul_overflow((size_t)a, (size_t)b, &n) || n > kMaxBytes / 2 - 256) return false;
  *out = (2 * n + 255) & ~(size_t)255;
  return true;
}

// Over more than one wave, 128 x 128 tiles are considered up to this many K
// steps: they move twice the operand bytes per product, and under long load
// the board's power limit makes that count for more than the estimates below
// say (8192 x 5120 x 17408, 640 large tiles or 2560: 1078 against 1499 us).
constexpr int64_t NARROW_STEPS = 16;

// K steps of a 128 x 128 tile that has a CU to itself, in 0.01 us: past
// LONG_RUN of them they cost `late`, not `step` (the operands then no longer
// come from the caches: A @ B.T 1664 x 1984 x 12672 117 us against 97 in
// parts of 256 x 256 tiles, x 8192 70 against 70).
constexpr int64_t LONG_RUN = 96;
int64_t narrow_steps(int64_t steps, int64_t step, int64_t late) {
  return steps <= LONG_RUN ? step * steps : step * LONG_RUN + late * (steps - LONG_RUN);
}

int64_t round8(int64_t x) { return (x + 7) & ~(int64_t)7; }

// Whether the LDS-DMA loads read a matrix in place: they need 4-byte
// addresses, and a range that ends between words (their range check is by
// word).  So rows of an even number of elements, at even distances.  Rows of
// K values in the small-output kernel (small_k): a multiple of 8, as it reads
// the last 16-byte piece whole.
bool direct(const void* p, int64_t ld, int64_t stride, int64_t cols, bool small_k) {
  return ((uintptr_t)p & 3) == 0 && ((ld | stride) & 1) == 0 && (cols & (small_k ? 7 : 1)) == 0;
}

// A matrix of the epilogue: its leading dimension and alignment.
dense_gemm_status check_matrix(const void* p, int64_t ld, int64_t N) {
  if (p == nullptr) return DENSE_GEMM_OK;
  if (ld < N) return DENSE_GEMM_BAD_LD;
  if (ld >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  return ((uintptr_t)p & 1) != 0 ? DENSE_GEMM_MISALIGNED : DENSE_GEMM_OK;
}

dense_gemm_status check_groups(const dense_gemm_groups* g) {
  if (g->count < 0) return DENSE_GEMM_INVALID_DIM;
  if (g->count >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  if (g->stride < 0) return DENSE_GEMM_BAD_ARG;
  // elements from the first group's matrix to the last's
  int64_t span;
  if (__builtin_mul_overflow(g->count, g->stride, &span) || span >= (int64_t)1 << 61)
    return DENSE_GEMM_TOO_LARGE;
  return DENSE_GEMM_OK;
}

// An upper bound on the row tiles of M rows in `count` groups: a group of m
// rows has at most (m + tile - 1) / tile, and at most min(count, M) groups
// have rows.
int64_t most_row_tiles(int64_t M, int64_t count, int64_t tile) {
  const int64_t active = count < M ? count : M;
  return (M + (tile - 1) * active) / tile;
}

}  // namespace

dense_gemm_status layer_validate(int op, int64_t M, int64_t N, int64_t K, const void* A,
                                 int64_t lda, const void* B, int64_t ldb, const void* D,
                                 int64_t ldd, const dense_gemm_epilogue* e,
                                 const dense_gemm_groups* g, bool* done) {
  *done = true;
  if (!valid_op(op)) return DENSE_GEMM_BAD_ARG;
  if (M < 0 || N < 0 || K < 0) return DENSE_GEMM_INVALID_DIM;
  dense_gemm_status st;
  // (without groups there is nothing to do, and an empty stack of matrices
  // has no pointer)
  if (g == nullptr || g->count != 0) {
    st = dense_gemm_validate(op_layout(op), M, N, K, A, lda, B, ldb, D, ldd);
    if (st != DENSE_GEMM_OK) return st;
  }
  if (e != nullptr) {
    if (e->act < DENSE_GEMM_ACT_NONE || e->act > DENSE_GEMM_ACT_SILU || (e->grad & ~1) != 0)
      return DENSE_GEMM_BAD_ARG;
    if (e->grad != 0 &&
        (e->act == DENSE_GEMM_ACT_NONE || e->bias != nullptr || e->residual != nullptr))
      return DENSE_GEMM_BAD_ARG;
    if (e->bias != nullptr && e->bias_stride < 0) return DENSE_GEMM_BAD_ARG;
  }
  if (g != nullptr) {
    st = check_groups(g);
    if (st != DENSE_GEMM_OK) return st;
    if (g->count > kLayerMaxGroups) return DENSE_GEMM_TOO_LARGE;
  }
  if (M == 0 || N == 0 || (g != nullptr && g->count == 0)) return DENSE_GEMM_OK;
  if (M > kLayerMaxDim || N > kLayerMaxDim || K > kLayerMaxDim) return DENSE_GEMM_TOO_LARGE;
  const int64_t tile = BM / 2;  // the smallest of the tiled kernels
  if (((M + tile - 1) / tile) * ((N + tile - 1) / tile) > kLayerMaxTiles) return DENSE_GEMM_TOO_LARGE;
  if (e != nullptr) {
    if (e->grad != 0 && e->preact == nullptr) return DENSE_GEMM_NULL_PTR;
    if (((uintptr_t)e->bias & 1) != 0) return DENSE_GEMM_MISALIGNED;
    st = check_matrix(e->residual, e->ldr, N);
    if (st != DENSE_GEMM_OK) return st;
    st = check_matrix(e->preact, e->ldz, N);
    if (st != DENSE_GEMM_OK) return st;
  }
  if (g != nullptr) {
    if (g->ends == nullptr) return DENSE_GEMM_NULL_PTR;
    if (((uintptr_t)g->ends & 3) != 0) return DENSE_GEMM_MISALIGNED;
    // the smallest tiles there are
    if (most_row_tiles(M, g->count, SMALL_TILE) * ((N + SMALL_TILE - 1) / SMALL_TILE) > kLayerMaxTiles)
      return DENSE_GEMM_TOO_LARGE;
  }
  *done = false;
  return DENSE_GEMM_OK;
}

// 128 x 128 tiles where they are estimated faster than the plain product's
// plan.  The estimates, in 0.01 us, are fitted to times on the MI355X (BF16,
// SILU in the epilogue, operands from HBM), nk K steps of 64:
//   * 256 x 256 tiles: waves x (133 nk + 1650); a split (choose_split) costs
//     800 and 4 per partial tile, a split last wave 1500;
//   * 256 x 128 and 128 x 256: waves x (75 nk + 960), a split 600 and 1.5 a
//     partial tile;
//   * 128 x 128, two workgroups per CU: waves x (79 nk + 650); where each has
//     a CU to itself 35 (A @ B.T) or 41 nk (later steps 90) + 550, and split-K
//     costs 600 and 1 per partial tile.
// Measured, us, the plain product's plan against 128 x 128: A @ B.T 2048 x
// 2048 x 2048 30 against 21, 777 x 1000 x 2048 29 against 19, 4096 x 2048 x
// 1024 22 against 20, x 4096 56 against 57, 4096 x 4096 x 512 27 against 25;
// A @ B 2048 x 2048 x 2048 51 against 23, 4096 x 2048 x 4096 88 against 60,
// 512 x 512 x 4096 29 against 18 (in 8 parts), 100 x 8000 x 3000 25 against 21.
// One tile row or column over several waves: 128 x 200000 x 512 80 against 64
// (A @ B 79 and 64), 128 x 70000 x 1024 53 and 47, 150000 x 64 x 256 41 and
// 27; A @ B 128 x 128256 x 1024, two full waves either way, 63 and 65.
dense_gemm_status layer_plan(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                             int64_t lda, const void* B, int64_t ldb, int64_t cus, CallPlan* cp) {
  const dense_gemm_status st = plan_call(layout, M, N, K, A, lda, B, ldb, cus, nullptr, cp);
  if (st != DENSE_GEMM_OK) return st;
  // (the plain product reads fewer operands in place)
  if (direct(A, lda, 0, K, cp->small())) {
    cp->a_direct = true;
    cp->a_bytes = 0;
  }
  if (direct(B, ldb, 0, layout == NT ? K : N, layout == NT && cp->small())) {
    cp->b_direct = true;
    cp->b_bytes = 0;
  }
  if (cp->small()) return st;
  const int64_t nk = (K + BK - 1) / BK;
  int64_t* plan = cp->plan;
  const int64_t had = plan[3] * plan[4], parts = cp->split_tiles * plan[8];
  const int64_t waves = (had + cus - 1) / cus;
  const bool large = plan[0] == BM && plan[1] == BN;
  const int64_t step0 = large ? 133 : 75, fixed0 = large ? 1650 : 960;
  double cost = (double)(plan[8] > 1 ? waves - 1 : waves) * (step0 * nk + fixed0);
  if (plan[8] > 1) {
    cost += step0 * plan[9] + fixed0;
    if (large)
      cost += had < cus ? 800 + 4.0 * parts : 1500;
    else
      cost += 600 + 1.5 * parts;
  }
  const int64_t tiles_m = (M + BM / 2 - 1) / (BM / 2), tiles_n = (N + BN / 2 - 1) / (BN / 2);
  const int64_t tasks = tiles_m * tiles_n, slots = cus * resident(BM / 2, BN / 2);
  int64_t splits = 1, steps = nk;
  const int64_t step = layout == NT ? 35 : 41;
  if (tasks < cus) choose_split(tasks, nk, cus, step, 600, 1, BM / 16, &splits, &steps);
  double narrow;
  if (splits > 1)
    narrow = (double)narrow_steps(steps, step, 90) + 1150 + splits * tasks;
  else if (tasks <= cus)
    narrow = (double)narrow_steps(nk, step, 90) + 550;
  else
    narrow = (double)((tasks + slots - 1) / slots) * (79 * nk + 650);
  if (narrow >= cost || (tasks > slots && nk > NARROW_STEPS)) return st;
  plan[0] = BM / 2;
  plan[1] = BN / 2;
  plan[3] = tiles_m;
  plan[4] = tiles_n;
  plan[5] = tasks * splits < slots ? tasks * splits : slots;
  plan[6] = choose_group_m(tiles_m);
  plan[7] = THREADS;
  plan[8] = splits;
  plan[9] = steps;
  cp->full_tasks = splits > 1 ? 0 : tasks;
  cp->split_tiles = tasks - cp->full_tasks;
  // (at most one part per CU: no overflow)
  cp->split_bytes =
      splits > 1 ? (size_t)(splits * tasks) * (BM / 2) * (BN / 2) * sizeof(float) : 0;
  return DENSE_GEMM_OK;
}

dense_gemm_status grouped_plan(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                               int64_t lda, const void* B, int64_t ldb, const dense_gemm_groups& g,
                               int64_t cus, GroupedPlan* out) {
  const int64_t K8 = round8(K), N8 = round8(N);
  // The ends are not known here: the tile follows the rows of an average
  // group (of those that can have any) and the number of tiles.  Measured
  // with BF16, us per call:
  //   * 256 x 256 against 128 x 128 tiles: 16 groups of 1024 rows, N = K =
  //     4096, 413 against 571; of 256 rows 191 against 201; 32 of 512, N =
  //     2048, 287 against 341; but 64 of 128 rows, N = K = 2048, 182 against
  //     161, and 16 of 128, N = K = 4096, 187 against 153.  Groups of more
  //     than 192 rows take 128 x 128 tiles too where their estimated time
  //     (that of layer_plan, half a tile of each group empty) is less: 4 of
  //     512, N = 512, K = 2048, 49 against 22; 16 of 512, N = K = 2048, 106
  //     against 80; of 2768, 328 against 392 (256 x 256 taken).  Over more
  //     than one round up to 32 K steps alone, as above.
  //   * A @ B also has 128 x 256 tiles (B's rows in longer pieces): 16 groups
  //     of 128 rows, N = K = 4096, 133 against 150 in 128 x 128 tiles, where
  //     they are enough for the CUs, or by the count estimated as above one
  //     round of them that fills three quarters: limits between the shapes
  //     measured here, with no model of the time behind them, and groups
  //     without rows count as ones with (8 unequal groups of 128, N = K =
  //     4096, 64 against 73; 32 of 128, N = 1024, K = 2048, 41 against 46); but 16 of
  //     64, N = K = 2048 (half the CUs), 38 against 30, 48 of 104, N = 1400, K
  //     = 1000 (1.5 rounds), 62 against 50.
  //   * The small-output kernel splits K among its waves, which pays where
  //     128 x 128 tiles would leave CUs idle or with one workgroup: A @ B.T
  //     with 8 groups of 1 to 16 rows, N = K = 4096 (256 such tiles), 42 to
  //     44 against 46 to 51; 32 groups, N = K = 2048 (512 tiles), 46 to 55
  //     against 46 to 47.  Its A @ B tiles read B in 32-byte pieces: 8 groups
  //     of one row, N = K = 4096, 51 against 44.
  const int64_t active = g.count < M ? g.count : M;
  const int64_t avg = (M + active - 1) / active;
  const int64_t tiles128 = most_row_tiles(M, g.count, BM / 2) * ((N + BN / 2 - 1) / (BN / 2));
  const int64_t nk = (K + BK - 1) / BK, slots128 = cus * resident(BM / 2, BN / 2);
  const int64_t est256 = (M + BM / 2 * active) / BM * ((N + BN - 1) / BN);
  const int64_t est128 = (M + BM / 4 * active) / (BM / 2) * ((N + BN / 2 - 1) / (BN / 2));
  const bool narrow = (est128 <= slots128 || nk <= 2 * NARROW_STEPS) &&
                      (double)((est128 + slots128 - 1) / slots128) * (79 * nk + 650) <
                          (double)((est256 + cus - 1) / cus) * (133 * nk + 1650);
  out->small = avg <= SMALL_TILE && tiles128 <= (layout == NT ? cus : cus / 4);
  if (out->small) {
    out->tile_m = out->tile_n = SMALL_TILE;
  } else if (avg > 192) {
    out->tile_m = narrow ? BM / 2 : BM;
    out->tile_n = narrow ? BN / 2 : BN;
  } else {
    out->tile_m = BM / 2;
    const int64_t rows = (M + BM / 4 * active) / (BM / 2), cols = (N + BN - 1) / BN;
    out->tile_n = layout == NN && ((M + BM / 2 - 1) / (BM / 2) * cols >= cus ||
                                   (rows * cols <= cus && 4 * rows * cols >= 3 * cus))
                      ? BN : BN / 2;
  }
  out->tiles_n = (N + out->tile_n - 1) / out->tile_n;
  const int64_t most = most_row_tiles(M, g.count, out->tile_m) * out->tiles_n;
  const int64_t slots = cus * resident(out->tile_m, out->tile_n);
  out->grid = out->small || most < slots ? most : slots;
  out->a_direct = K == 0 || direct(A, lda, 0, K, out->small);
  out->matrices = g.stride == 0 ? 1 : g.count;
  out->b_direct = K == 0 || direct(B, ldb, g.stride, layout == NT ? K : N, layout == NT && out->small);
  out->a_bytes = out->b_bytes = 0;
  if (!out->a_direct && !matrix_bytes(M, K8, &out->a_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (!out->b_direct) {
    int64_t rows;
    if (__builtin_mul_overflow(out->matrices, layout == NT ? N : K, &rows) ||
        !matrix_bytes(rows, layout == NT ? K8 : N8, &out->b_bytes))
      return DENSE_GEMM_TOO_LARGE;
  }
  return DENSE_GEMM_OK;
}

dense_gemm_status tn_validate(int fmt, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* B, int64_t ldb, const void* D, int64_t ldd,
                              const void* colsum, const dense_gemm_groups* g, bool* done) {
  *done = true;
  if (fmt != DENSE_GEMM_F16 && fmt != DENSE_GEMM_BF16) return DENSE_GEMM_BAD_ARG;
  if (M < 0 || N < 0 || K < 0) return DENSE_GEMM_INVALID_DIM;
  if (g != nullptr) {
    const dense_gemm_status st = check_groups(g);
    if (st != DENSE_GEMM_OK) return st;
  }
  const int64_t groups = g != nullptr ? g->count : 1;
  if (M == 0 || groups == 0) return DENSE_GEMM_OK;
  if (N == 0) return colsum != nullptr ? DENSE_GEMM_BAD_ARG : DENSE_GEMM_OK;
  if (M > kLayerMaxDim || N > kLayerMaxDim || K > kLayerMaxDim) return DENSE_GEMM_TOO_LARGE;
  int64_t tasks;
  const int64_t tile = BM / 2;  // the smaller
  if (__builtin_mul_overflow(((M + tile - 1) / tile) * ((N + tile - 1) / tile), groups, &tasks) ||
      tasks > kLayerMaxTiles)
    return DENSE_GEMM_TOO_LARGE;
  // and the blocks of 16 column sums each
  if (colsum != nullptr &&
      (__builtin_mul_overflow((M + 15) / 16, groups, &tasks) || tasks > kLayerMaxTiles))
    return DENSE_GEMM_TOO_LARGE;
  if (D == nullptr || (K > 0 && (A == nullptr || B == nullptr))) return DENSE_GEMM_NULL_PTR;
  if (ldd < N || (K > 0 && (lda < M || ldb < N))) return DENSE_GEMM_BAD_LD;
  if (((uintptr_t)D & 1) != 0 || ((uintptr_t)colsum & 1) != 0) return DENSE_GEMM_MISALIGNED;
  if (ldd >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  if (K > 0) {
    if (((uintptr_t)A & 1) != 0 || ((uintptr_t)B & 1) != 0) return DENSE_GEMM_MISALIGNED;
    if (lda >= kMaxDim || ldb >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
    // 32-bit buffer offsets: the rows of one K step, as given or repacked
    const int64_t lim = ((int64_t)1 << 31) - 16;
    const int64_t M8 = round8(M), N8 = round8(N);
    if (((BK - 1) * (lda > M8 ? lda : M8) + M8) * 2 >= lim) return DENSE_GEMM_TOO_LARGE;
    if (((BK - 1) * (ldb > N8 ? ldb : N8) + N8) * 2 >= lim) return DENSE_GEMM_TOO_LARGE;
  }
  if (g != nullptr) {
    if (g->ends == nullptr) return DENSE_GEMM_NULL_PTR;
    if (((uintptr_t)g->ends & 3) != 0) return DENSE_GEMM_MISALIGNED;
    if (groups > 1 && g->stride < (M - 1) * ldd + N) return DENSE_GEMM_BAD_LD;
  }
  *done = false;
  return DENSE_GEMM_OK;
}

// Column sums: up to this many K steps the first tile of each tile row adds
// its columns alone; beyond, the row's tiles share the steps and a second
// kernel adds up theirs (layer_kernel.h).  Measured, us, alone against shared:
// 1024 x 1024 x 333 8.5 and 14.9, 5120 x 8192 x 1024 87 and 90, x 8192 532 and
// 530; 64 groups, 2048 x 2048 each, of 64 rows 136 and 150; 16 of 4096 rows,
// 512 x 512, 67 and 64.  Groups may be several times as long as their average,
// which is all that is known here, and the longest decide: they count four
// times (16 unevenly filled groups of 1024 rows on average, 4096 x
// 4096, 535 and 519).
constexpr int64_t DIRECT_SUM_STEPS = 32;

// One way to run D = A.T @ B, and its estimated time in 0.01 us, by a model
// fitted to times on the MI355X (BF16):
//   * 256 x 256 tiles, one workgroup per CU: waves x (133 per K step + 850);
//     split-K as for the other products (choose_split: 105, 1200, 12; a split
//     last wave costs 2500 on top of its steps);
//   * 128 x 128 tiles, two per CU: waves x (90 per K step + 360), or 47 per
//     step (later ones 70) + 550 where each has a CU to itself; split-K only
//     then (600 for the second kernel, 1 per partial tile).
// Measured 256 against 128, us: 4096 x 4096 x 2048 64 against 69; 4096 x 2304
// x 4096 93 against 111, 4096 x 2048 x 4096 93 against 64 (512 of the smaller
// tiles: just one wave); 2048 x 2048 x 8192 in 4 parts 77 against 73; 512 x
// 640 x 20011 in 32 parts 38, in 12 parts of the smaller 26; 40 groups of 75
// rows, 520 x 1000, 25 against 20; 16 of 1024, 4096 x 4096, 483 against 593.
struct TnChoice {
  int64_t tile, splits, steps;
  double cost;
};

static TnChoice tn_choice(int64_t M, int64_t N, int64_t nk, int64_t groups, bool grouped,
                          int64_t cus, int64_t tile) {
  TnChoice c = {tile, 1, nk, 0.0};
  const int64_t tasks = ((M + tile - 1) / tile) * ((N + tile - 1) / tile) * groups;
  const int64_t slots = cus * resident(tile, tile);
  const int64_t waves = (tasks + slots - 1) / slots;
  // Parts against few tiles.  With groups they also even out the groups'
  // lengths, so they are chosen as for a group of twice the average; a last
  // wave is not split (which tiles it holds is not known here).
  const int64_t reach = grouped ? 2 * nk : nk;
  if (tile == BM) {
    const int64_t last = tasks % cus;
    if (!grouped || tasks < cus)
      choose_split(tasks, reach, cus, 105, 1200, 12, BM / 16, &c.splits, &c.steps);
    c.cost = (double)waves * (133 * nk + 850);
    if (c.splits > 1)
      c.cost = (double)(waves - 1) * (133 * nk + 850) + 133 * ((nk + c.splits - 1) / c.splits) + 850 + 2500 +
               (tasks < cus ? 12 * c.splits * last - 1300 : 0);
  } else if (tasks < cus) {
    choose_split(tasks, reach, cus, 47, 600, 1, BM / 16, &c.splits, &c.steps);
    c.cost = narrow_steps((nk + c.splits - 1) / c.splits, 47, 70) + 550 +
             (c.splits > 1 ? 600 + c.splits * tasks : 0);
  } else {
    c.cost = (double)waves * (90 * nk + 360);
    if (waves > 1 && nk > NARROW_STEPS) c.cost = 1e30;
  }
  return c;
}

dense_gemm_status tn_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                          const void* B, int64_t ldb, bool colsum, const dense_gemm_groups* g,
                          int64_t cus, TnPlan* out) {
  out->groups = g != nullptr ? g->count : 1;
  // With groups, the plan is made for groups of average length (of those
  // that can have rows).
  int64_t rows = K;
  if (g != nullptr) {
    const int64_t active = g->count < K ? g->count : K;
    rows = active > 0 ? (K + active - 1) / active : 0;
  }
  const int64_t nk = (rows + BK - 1) / BK;
  const TnChoice wide = tn_choice(M, N, nk, out->groups, g != nullptr, cus, BM);
  const TnChoice narrow = tn_choice(M, N, nk, out->groups, g != nullptr, cus, BM / 2);
  const TnChoice& best = narrow.cost < wide.cost ? narrow : wide;
  out->tile = best.tile;
  out->tiles_m = (M + best.tile - 1) / best.tile;
  out->tiles_n = (N + best.tile - 1) / best.tile;
  out->splits = best.splits;
  out->steps = best.steps;
  const int64_t tasks = out->tiles_m * out->tiles_n * out->groups;
  out->full_tasks = best.splits == 1 ? tasks : tasks < cus ? 0 : tasks - tasks % cus;
  out->split_tiles = tasks - out->full_tasks;
  out->a_direct = K == 0 || direct(A, lda, 0, M, false);
  out->b_direct = K == 0 || direct(B, ldb, 0, N, false);
  out->a_bytes = out->b_bytes = out->split_bytes = out->sums_bytes = 0;
  if (!out->a_direct && !matrix_bytes(K, round8(M), &out->a_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (!out->b_direct && !matrix_bytes(K, round8(N), &out->b_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (out->splits > 1) {
    // (at most one part per resident workgroup: no overflow)
    out->split_bytes =
        (size_t)(out->splits * out->split_tiles) * out->tile * out->tile * sizeof(float);
  }
  if (colsum && !(out->splits == 1 && (g != nullptr ? 4 * nk : nk) <= DIRECT_SUM_STEPS))
    out->sums_bytes = (size_t)(out->full_tasks + out->splits * out->split_tiles) * 2 * out->tile *
                      sizeof(float);
  return DENSE_GEMM_OK;
}

}  // namespace dg
