// grouped.hip -- dense_gemm_layer with row groups (include/dense_gemm.h):
// the products of a mixture of experts, D[rows of g] = epilogue(A[rows of g]
// @ Bhat_g) for the rows of every group g, on the MI355X (gfx950).  Host
// side: the plan (grouped_plan in plan_layer.cpp) and the launches.  The
// kernels find their tiles' groups on the device (groups.h).
#include "layer_host.h"

namespace dg {

template <typename T, int LAYOUT>
dense_gemm_status run_grouped(LayerCall c, const dense_gemm_groups& groups, void* ws,
                              size_t ws_bytes) {
  GroupedPlan gp;
  const dense_gemm_status st = grouped_plan(LAYOUT, c.M, c.N, c.K, c.A, c.lda, c.B, c.ldb, groups,
                                            c.cus, &gp);
  if (st != DENSE_GEMM_OK) return st;
  if (gp.total() > 0) {
    if (ws == nullptr || ws_bytes < gp.total()) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)ws & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  Groups g = {(const int32_t*)groups.ends, (int)groups.count, (int)c.M, groups.stride};
  const int64_t b_rows = LAYOUT == NT ? c.N : c.K;
  // (one matrix for all groups is copied once, and stays one)
  repack_operands(c, gp.a_direct ? nullptr : ws, gp.matrices, b_rows, LAYOUT == NT ? c.K : c.N,
                  g.stride, gp.b_direct ? nullptr : (char*)ws + gp.a_bytes);
  if (!gp.b_direct && gp.matrices > 1) g.stride = b_rows * c.ldb;
  const dim3 grid((unsigned)gp.grid);
  if (gp.small) {
    SmallLayerParams p = small_params(c);
    p.tiles_n = (int)gp.tiles_n;
    p.g = g;
    hipLaunchKernelGGL((gemm_small<T, LAYOUT, 1, 1, true, true>), grid, dim3(SMALL_THREADS), 0,
                       c.stream, p);
    return launched();
  }
  LayerParams p = {};
  set_operands(p, c);
  p.tiles_n = (int)gp.tiles_n;
  p.group_m = choose_group_m(kMaxDim);
  p.e = device_epilogue(c.e);
  p.g = g;
  if (gp.tile_n == BN / 2) {
    hipLaunchKernelGGL((layer_gemm_kernel<T, LAYOUT, false, BN / 2, BM / 2, true>), grid,
                       dim3(THREADS), 0, c.stream, p);
    return launched();
  }
  if constexpr (LAYOUT == NN) {
    if (gp.tile_m == BM / 2) {
      hipLaunchKernelGGL((layer_gemm_kernel<T, LAYOUT, false, BN, BM / 2, true>), grid, dim3(THREADS),
                         0, c.stream, p);
      return launched();
    }
  }
  hipLaunchKernelGGL((layer_gemm_kernel<T, LAYOUT, false, BN, BM, true>), grid, dim3(THREADS), 0,
                     c.stream, p);
  return launched();
}

template dense_gemm_status run_grouped<_Float16, NT>(LayerCall, const dense_gemm_groups&, void*, size_t);
template dense_gemm_status run_grouped<_Float16, NN>(LayerCall, const dense_gemm_groups&, void*, size_t);
template dense_gemm_status run_grouped<__bf16, NT>(LayerCall, const dense_gemm_groups&, void*, size_t);
template dense_gemm_status run_grouped<__bf16, NN>(LayerCall, const dense_gemm_groups&, void*, size_t);

}  // namespace dg
