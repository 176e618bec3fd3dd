// tn.hip -- a layer's weight and bias gradients on the MI355X (gfx950): D =
// A.T @ B and the column sums of A, for one matrix or one per group of rows
// (dense_gemm_tn, include/dense_gemm.h).  Host side: the plan (tn_plan in
// plan_layer.cpp), the launches and the C ABI entry points.  The kernel is
// the tiled one with layout TA (layer_kernel.h): A and B both have k as their
// row, so their tiles are 64 k rows and both operands' MFMA
// fragments come from transposing LDS reads.
#include "column_sums.h"
#include "layer_host.h"
#include "split_reduce.h"

namespace dg {

template <typename T, int TILE, bool GROUP, bool SUMS>
static void enqueue_tile(const LayerParams& p, const ColumnSumsParams& sums, int64_t sums_blocks,
                         int cus, hipStream_t stream) {
  const int slots = cus * (int)resident(TILE, TILE);
  const dim3 grid((unsigned)(p.num_tasks < slots ? p.num_tasks : slots)), block(THREADS);
  if (p.splits > 1 || (resident(TILE, TILE) > 1 && p.num_tasks <= cus))
    // (whole 128 x 128 tiles that have a CU each also run this kernel, for
    // its deeper rings)
    hipLaunchKernelGGL((layer_gemm_kernel<T, TA, true, TILE, TILE, GROUP, SUMS>), grid, block, 0,
                       stream, p);
  else
    hipLaunchKernelGGL((layer_gemm_kernel<T, TA, false, TILE, TILE, GROUP, SUMS>), grid, block, 0,
                       stream, p);
  if (p.splits > 1) {
    LayerReduceParams r = {};
    (ReduceParams&)r = {p.D, p.ws, p.M, p.N, p.ldd, p.tiles_m, p.tiles_n, p.group_m,
                        p.full_tasks, p.splits, p.tiles, 1};
    r.stride = p.g.stride;
    r.sums = sums;
    r.sums_blocks = sums_blocks;
    enqueue_split_reduce<T, TILE, TILE>(r, cus, stream);
  } else if (SUMS && p.colsum_ws != nullptr) {
    const int64_t grid = sums_blocks < CS_MAX_GRID ? sums_blocks : CS_MAX_GRID;
    hipLaunchKernelGGL((column_sums<T, TILE>), dim3((unsigned)grid), dim3(CS_THREADS), 0, stream, sums,
                       (int)sums_blocks);
  }
}

template <typename T, int TILE>
static dense_gemm_status enqueue_tn(const LayerParams& p, uint16_t* colsum, int groups, bool grouped,
                                    int cus, hipStream_t stream) {
  const ColumnSumsParams s = {p.colsum_ws, colsum, p.M, groups, p.tiles_m, p.tiles_n, p.group_m,
                              p.full_tasks, p.splits, p.tiles};
  if (colsum == nullptr) {
    grouped ? enqueue_tile<T, TILE, true, false>(p, s, 0, cus, stream)
            : enqueue_tile<T, TILE, false, false>(p, s, 0, cus, stream);
  } else {
    const int64_t blocks = column_sums_blocks(p.M, groups);
    grouped ? enqueue_tile<T, TILE, true, true>(p, s, blocks, cus, stream)
            : enqueue_tile<T, TILE, false, true>(p, s, blocks, cus, stream);
  }
  return launched();
}

template <typename T>
static dense_gemm_status run_tn(LayerCall c, void* colsum, const dense_gemm_groups* groups,
                                void* ws, size_t ws_bytes) {
  TnPlan tp;
  const dense_gemm_status st = tn_plan(c.M, c.N, c.K, c.A, c.lda, c.B, c.ldb, colsum != nullptr, groups,
                                       c.cus, &tp);
  if (st != DENSE_GEMM_OK) return st;
  if (tp.total() > 0) {
    if (ws == nullptr || ws_bytes < tp.total()) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)ws & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  char* at = (char*)ws;
  Repack a = {}, b = {};
  if (!tp.a_direct) {
    a = {c.A, at, 1, c.K, c.M, c.lda, 0};
    c.A = (const uint16_t*)at;
    c.lda = repacked_ld(c.M);
  }
  at += tp.a_bytes;
  if (!tp.b_direct) {
    b = {c.B, at, 1, c.K, c.N, c.ldb, 0};
    c.B = (const uint16_t*)at;
    c.ldb = repacked_ld(c.N);
  }
  at += tp.b_bytes;
  enqueue_repacks(a, b, c.stream);
  LayerParams p = {};
  set_operands(p, c);
  p.tiles_m = (int)tp.tiles_m;
  p.tiles_n = (int)tp.tiles_n;
  p.group_m = choose_group_m(tp.tiles_m);
  p.full_tasks = (int)tp.full_tasks;
  p.tiles = (int)tp.split_tiles;
  p.splits = (int)tp.splits;
  p.split_steps = (int)tp.steps;
  p.num_tasks = (int)(tp.full_tasks + tp.split_tiles * tp.splits);
  if (tp.splits > 1) p.ws = (float*)at;
  if (tp.sums_bytes > 0) p.colsum_ws = (float*)(at + tp.split_bytes);
  p.colsum = (uint16_t*)colsum;
  if (groups != nullptr)
    p.g = {(const int32_t*)groups->ends, (int)groups->count, (int)c.K, groups->stride};
  return tp.tile == BM ? enqueue_tn<T, BM>(p, (uint16_t*)colsum, (int)tp.groups, groups != nullptr,
                                           c.cus, c.stream)
                       : enqueue_tn<T, BM / 2>(p, (uint16_t*)colsum, (int)tp.groups,
                                               groups != nullptr, c.cus, c.stream);
}

}  // namespace dg

using namespace dg;

extern "C" {

dense_gemm_status dense_gemm_tn(int fmt, int64_t M, int64_t N, int64_t K, const void* A,
                                int64_t lda, const void* B, int64_t ldb, void* D, int64_t ldd,
                                void* colsum, const dense_gemm_groups* groups, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  bool done;
  dense_gemm_status st = tn_validate(fmt, M, N, K, A, lda, B, ldb, D, ldd, colsum, groups, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  LayerCall c = {M, N, K, (const uint16_t*)A, lda, (const uint16_t*)B, ldb, (uint16_t*)D, ldd,
                 nullptr, 0, 1, stream};
  st = device_topology(&c.cus, &c.xcds);
  if (st != DENSE_GEMM_OK) return st;
  return fmt == DENSE_GEMM_BF16 ? run_tn<__bf16>(c, colsum, groups, workspace, workspace_bytes)
                                : run_tn<_Float16>(c, colsum, groups, workspace, workspace_bytes);
}

dense_gemm_status dense_gemm_tn_workspace_size(int64_t M, int64_t N, int64_t K, const void* A,
                                               int64_t lda, const void* B, int64_t ldb, int colsum,
                                               const dense_gemm_groups* groups, int64_t num_cus,
                                               size_t* bytes) {
  if (bytes == nullptr || num_cus < 0) return DENSE_GEMM_BAD_ARG;
  const void* any = (const void*)(uintptr_t)16;
  dense_gemm_groups g = {any, 0, 0};
  if (groups != nullptr) {
    g.count = groups->count;
    // (the stride concerns D alone: any that keeps the outputs apart will do)
    if (M > 0 && N > 0 && M < kMaxDim && N < kMaxDim) g.stride = M * N;
  }
  bool done;
  dense_gemm_status st = tn_validate(DENSE_GEMM_F16, M, N, K, A, lda, B, ldb, any, N,
                                     colsum != 0 ? any : nullptr, groups != nullptr ? &g : nullptr,
                                     &done);
  if (st != DENSE_GEMM_OK) return st;
  *bytes = 0;
  if (done) return DENSE_GEMM_OK;
  int cus = (int)(num_cus < kMaxDim ? num_cus : kMaxDim - 1), xcds;
  if (num_cus == 0) {
    st = device_topology(&cus, &xcds);
    if (st != DENSE_GEMM_OK) return st;
  }
  TnPlan tp;
  st = tn_plan(M, N, K, A, lda, B, ldb, colsum != 0, groups != nullptr ? &g : nullptr, cus, &tp);
  if (st == DENSE_GEMM_OK) *bytes = tp.total();
  return st;
}

}  // extern "C"
