// layer.hip -- the products of a transformer layer on the MI355X (gfx950):
// the FP16/BF16 product with bias, activation and residual in its epilogue
// and its gradient form (dense_gemm_layer, include/dense_gemm.h).  Host side:
// the plan (layer_plan in plan_layer.cpp), the launches and the C ABI entry
// point, which hands calls with row groups to grouped.hip.  The kernels are
// layer_gemm_kernel (layer_kernel.h) and, for small outputs, gemm_small with
// the epilogue of epilogue.h.
#include "layer_host.h"
#include "repack.h"
#include "split_reduce.h"

namespace dg {

void enqueue_repacks(const Repack& a, const Repack& b, hipStream_t stream) {
  const Repack* in[2] = {&a, &b};
  RepackJob job[2] = {};
  int64_t grid = 0;
  for (int i = 0; i < 2; ++i) {
    const Repack& r = *in[i];
    if (r.dst == nullptr) continue;
    RepackJob& j = job[i];
    j = {(const uint16_t*)r.src, (uint16_t*)r.dst, r.count, r.rows, r.cols, r.ld, r.stride,
         repacked_ld(r.cols), 0, 1};
    while (j.lanes < 256 && j.lanes * 8 < j.dcols) j.lanes *= 2;
    const int64_t per = 256 / j.lanes;
    j.blocks = (r.count * r.rows + per - 1) / per;
    if (j.blocks > REPACK_GROUPS_MAX_BLOCKS) j.blocks = REPACK_GROUPS_MAX_BLOCKS;
    grid += j.blocks;
  }
  if (grid > 0)
    hipLaunchKernelGGL(repack_groups, dim3((unsigned)grid), dim3(256), 0, stream, job[0], job[1]);
}

template <typename T, int LAYOUT, int TN, int TM>
static dense_gemm_status enqueue_tiled(const LayerCall& c, const CallPlan& cp, float* parts) {
  LayerParams p = {};
  set_operands(p, c);
  p.tiles_m = (int)cp.plan[3];
  p.tiles_n = (int)cp.plan[4];
  p.group_m = (int)cp.plan[6];
  p.full_tasks = (int)cp.full_tasks;
  p.tiles = (int)cp.split_tiles;
  p.splits = (int)cp.plan[8];
  p.split_steps = (int)cp.plan[9];
  p.num_tasks = (int)(cp.full_tasks + cp.split_tiles * cp.plan[8]);
  p.ws = parts;
  p.e = device_epilogue(c.e);
  const int slots = c.cus * (int)resident(TM, TN);
  const dim3 grid((unsigned)(p.num_tasks < slots ? p.num_tasks : slots)), block(THREADS);
  if (p.splits > 1 || (resident(TM, TN) > 1 && p.num_tasks <= c.cus)) {
    // (whole 128 x 128 tiles that have a CU each also run this kernel, for
    // its deeper rings)
    hipLaunchKernelGGL((layer_gemm_kernel<T, LAYOUT, true, TN, TM, false>), grid, block, 0, c.stream, p);
    if (p.splits == 1) return launched();
    LayerReduceParams r = {};
    (ReduceParams&)r = {p.D, p.ws, p.M, p.N, p.ldd, p.tiles_m, p.tiles_n, p.group_m,
                        p.full_tasks, p.splits, p.tiles, 1};
    r.e = p.e;
    enqueue_split_reduce<T, TN, TM>(r, c.cus, c.stream);
  } else {
    hipLaunchKernelGGL((layer_gemm_kernel<T, LAYOUT, false, TN, TM, false>), grid, block, 0, c.stream, p);
  }
  return launched();
}

template <typename T, int LAYOUT>
static dense_gemm_status enqueue_small_output(const LayerCall& c, const CallPlan& cp) {
  SmallLayerParams p = small_params(c);
  p.tiles_m = (int)cp.plan[3];
  p.tiles_n = (int)cp.plan[4];
  const dim3 grid((unsigned)(cp.plan[3] * cp.plan[4])), block(SMALL_THREADS);
  if constexpr (LAYOUT == NT) {
    if (cp.plan[0] == 2 * SMALL_TILE) {
      if (cp.plan[1] == 2 * SMALL_TILE)
        hipLaunchKernelGGL((gemm_small<T, LAYOUT, 2, 2, true>), grid, block, 0, c.stream, p);
      else
        hipLaunchKernelGGL((gemm_small<T, LAYOUT, 2, 1, true>), grid, block, 0, c.stream, p);
      return launched();
    }
  }
  hipLaunchKernelGGL((gemm_small<T, LAYOUT, 1, 1, true>), grid, block, 0, c.stream, p);
  return launched();
}

template <typename T, int LAYOUT>
static dense_gemm_status run_layer(LayerCall c, void* ws, size_t ws_bytes) {
  CallPlan cp;
  const dense_gemm_status st = layer_plan(LAYOUT, c.M, c.N, c.K, c.A, c.lda, c.B, c.ldb, c.cus, &cp);
  if (st != DENSE_GEMM_OK) return st;
  if (cp.total() > 0) {
    if (ws == nullptr || ws_bytes < cp.total()) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)ws & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  char* at = (char*)ws;
  repack_operands(c, cp.a_direct ? nullptr : at, 1, LAYOUT == NT ? c.N : c.K,
                  LAYOUT == NT ? c.K : c.N, 0, cp.b_direct ? nullptr : at + cp.a_bytes);
  at += cp.a_bytes + cp.b_bytes;
  if (cp.small()) return enqueue_small_output<T, LAYOUT>(c, cp);
  const bool short_tiles = cp.plan[0] == BM / 2;
  if (short_tiles && cp.plan[1] == BN / 2)
    return enqueue_tiled<T, LAYOUT, BN / 2, BM / 2>(c, cp, (float*)at);
  if constexpr (LAYOUT == NT) {
    if (cp.plan[1] == BN / 2) return enqueue_tiled<T, LAYOUT, BN / 2, BM>(c, cp, (float*)at);
  }
  return short_tiles ? enqueue_tiled<T, LAYOUT, BN, BM / 2>(c, cp, (float*)at)
                     : enqueue_tiled<T, LAYOUT, BN, BM>(c, cp, (float*)at);
}

}  // namespace dg

using namespace dg;

extern "C" {

dense_gemm_status dense_gemm_layer(int op, int64_t M, int64_t N, int64_t K, const void* A,
                                   int64_t lda, const void* B, int64_t ldb, void* D, int64_t ldd,
                                   const dense_gemm_epilogue* epilogue,
                                   const dense_gemm_groups* groups, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  bool done;
  dense_gemm_status st = layer_validate(op, M, N, K, A, lda, B, ldb, D, ldd, epilogue, groups, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  LayerCall c = {M, N, K, (const uint16_t*)A, lda, (const uint16_t*)B, ldb, (uint16_t*)D, ldd,
                 epilogue, 0, 1, stream};
  st = device_topology(&c.cus, &c.xcds);
  if (st != DENSE_GEMM_OK) return st;
  const bool bf16 = op == DENSE_GEMM_NN_BF16 || op == DENSE_GEMM_NT_BF16;
  const bool nt = op_layout(op) == NT;
  if (groups != nullptr) {
    if (nt)
      return bf16 ? run_grouped<__bf16, NT>(c, *groups, workspace, workspace_bytes)
                  : run_grouped<_Float16, NT>(c, *groups, workspace, workspace_bytes);
    return bf16 ? run_grouped<__bf16, NN>(c, *groups, workspace, workspace_bytes)
                : run_grouped<_Float16, NN>(c, *groups, workspace, workspace_bytes);
  }
  if (nt)
    return bf16 ? run_layer<__bf16, NT>(c, workspace, workspace_bytes)
                : run_layer<_Float16, NT>(c, workspace, workspace_bytes);
  return bf16 ? run_layer<__bf16, NN>(c, workspace, workspace_bytes)
              : run_layer<_Float16, NN>(c, workspace, workspace_bytes);
}

dense_gemm_status dense_gemm_layer_workspace_size(int op, int64_t M, int64_t N, int64_t K,
                                                  const void* A, int64_t lda, const void* B,
                                                  int64_t ldb, const dense_gemm_groups* groups,
                                                  int64_t num_cus, size_t* bytes) {
  if (bytes == nullptr || num_cus < 0) return DENSE_GEMM_BAD_ARG;
  // (D and the ends are looked at no further than for null)
  const void* any = (const void*)(uintptr_t)16;
  dense_gemm_groups g = {any, 0, 0};
  if (groups != nullptr) {
    g.count = groups->count;
    g.stride = groups->stride;
  }
  bool done;
  dense_gemm_status st = layer_validate(op, M, N, K, A, lda, B, ldb, any, N, nullptr,
                                        groups != nullptr ? &g : nullptr, &done);
  if (st != DENSE_GEMM_OK) return st;
  *bytes = 0;
  if (done) return DENSE_GEMM_OK;
  int cus = (int)(num_cus < kMaxDim ? num_cus : kMaxDim - 1), xcds;
  if (num_cus == 0) {
    st = device_topology(&cus, &xcds);
    if (st != DENSE_GEMM_OK) return st;
  }
  if (groups != nullptr) {
    GroupedPlan gp;
    st = grouped_plan(op_layout(op), M, N, K, A, lda, B, ldb, g, cus, &gp);
    if (st == DENSE_GEMM_OK) *bytes = gp.total();
    return st;
  }
  CallPlan cp;
  st = layer_plan(op_layout(op), M, N, K, A, lda, B, ldb, cus, &cp);
  if (st == DENSE_GEMM_OK) *bytes = cp.total();
  return st;
}

}  // extern "C"
