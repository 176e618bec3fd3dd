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

int64_t round8(int64_t x) { return (x + 7) & ~(int64_t)7; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

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
  dense_gemm_status st = dense_gemm_validate(op_layout(op), M, N, K, A, lda, B, ldb, D, ldd);
  if (st != DENSE_GEMM_OK) return st;
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
  }
  if (M == 0 || N == 0 || (g != nullptr && g->count == 0)) return DENSE_GEMM_OK;
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
    // tile numbers are 32-bit: the smallest tiles there are
    if (most_row_tiles(M, g->count, SMALL_TILE) * ((N + SMALL_TILE - 1) / SMALL_TILE) >= kMaxDim)
      return DENSE_GEMM_TOO_LARGE;
  }
  *done = false;
  return DENSE_GEMM_OK;
}

dense_gemm_status grouped_plan(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                               int64_t lda, const void* B, int64_t ldb, const dense_gemm_groups& g,
                               int64_t cus, GroupedPlan* out) {
  const int64_t K8 = round8(K), N8 = round8(N);
  // The ends are not known here: the tile follows the rows of an average
  // group (of those that can have any).
  const int64_t active = g.count < M ? g.count : M;
  const int64_t avg = (M + active - 1) / active;
  out->small = avg <= SMALL_TILE;
  if (out->small) {
    out->tile_m = out->tile_n = SMALL_TILE;
  } else {
    out->tile_m = avg <= 192 ? BM / 2 : BM;
    out->tile_n = BN;
  }
  out->tiles_n = (N + out->tile_n - 1) / out->tile_n;
  const int64_t most = most_row_tiles(M, g.count, out->tile_m) * out->tiles_n;
  out->grid = out->small || most < cus ? most : cus;
  out->a_direct = K == 0 || (aligned16(A) && (lda & 7) == 0 && (K & 7) == 0);
  out->b_direct = K == 0 || (aligned16(B) && (ldb & 7) == 0 && (g.stride & 7) == 0 &&
                             ((layout == NT ? K : N) & 7) == 0);
  out->a_bytes = out->b_bytes = 0;
  if (!out->a_direct && !matrix_bytes(M, K8, &out->a_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (!out->b_direct) {
    int64_t rows;
    if (__builtin_mul_overflow(g.count, layout == NT ? N : K, &rows) ||
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
  if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  // task numbers are 32-bit
  int64_t tasks;
  if (__builtin_mul_overflow(((M + BM - 1) / BM) * ((N + BN - 1) / BN), groups, &tasks) ||
      tasks >= kMaxDim)
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

dense_gemm_status tn_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                          const void* B, int64_t ldb, const dense_gemm_groups* g, int64_t cus,
                          TnPlan* out) {
  out->tiles_m = (M + BM - 1) / BM;
  out->tiles_n = (N + BN - 1) / BN;
  out->groups = g != nullptr ? g->count : 1;
  const int64_t tasks = out->tiles_m * out->tiles_n * out->groups;
  // Split-K by the tiled kernel's model (choose_split).  With groups, the
  // parts are chosen for a group of average length, and only where there are
  // fewer tiles than CUs: how the tiles' work falls on a last wave is not
  // known here.
  int64_t rows = K;
  if (g != nullptr) {
    const int64_t active = g->count < K ? g->count : K;
    rows = active > 0 ? (K + active - 1) / active : 0;
  }
  const int64_t nk = (rows + BK - 1) / BK;
  out->splits = 1;
  out->steps = nk;
  if (g == nullptr || tasks < cus)
    choose_split(tasks, nk, cus, 105, 1200, 12, BM / 16, &out->splits, &out->steps);
  out->full_tasks = tasks;
  if (out->splits > 1) out->full_tasks = tasks < cus ? 0 : tasks - tasks % cus;
  out->split_tiles = tasks - out->full_tasks;
  out->a_direct = K == 0 || (aligned16(A) && (lda & 7) == 0 && (M & 7) == 0);
  out->b_direct = K == 0 || (aligned16(B) && (ldb & 7) == 0 && (N & 7) == 0);
  out->a_bytes = out->b_bytes = out->split_bytes = out->sums_bytes = 0;
  if (!out->a_direct && !matrix_bytes(K, round8(M), &out->a_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (!out->b_direct && !matrix_bytes(K, round8(N), &out->b_bytes)) return DENSE_GEMM_TOO_LARGE;
  if (out->splits > 1) {
    // (at most one part per CU: no overflow)
    out->split_bytes = (size_t)(out->splits * out->split_tiles) * BM * BN * sizeof(float);
    out->sums_bytes = (size_t)(out->splits * out->split_tiles) * BM * sizeof(float);
  }
  return DENSE_GEMM_OK;
}

}  // namespace dg
