// plan_layer.h -- host-side planning of a layer's products (plain C++, no
// device code): the argument checks of dense_gemm_layer and dense_gemm_tn,
// their launch plans and the workspace they need.  Implemented in
// plan_layer.cpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan.h"

namespace dg {

// Workgroups that a CU holds at a time: the kernels with 128 x 128 tiles are
// built for two.
constexpr int64_t resident(int64_t tile_m, int64_t tile_n) {
  return tile_m == BM / 2 && tile_n == BN / 2 ? 2 : 1;
}

// The kernels count rows, columns, K and tasks in 32 bits and look a tile's
// height, a few K steps or one round of workgroups past the end.
constexpr int64_t kLayerMaxDim = kMaxDim - 1024;
constexpr int64_t kLayerMaxTiles = kMaxDim - (1 << 20);
// Every workgroup walks the ends of the groups past those held in registers
// (groups.h) twice, 64 at a time: about 0.03 us a group, so no array of ends
// takes longer than some 35 ms to search.
constexpr int64_t kLayerMaxGroups = 1 << 20;

// A call of dense_gemm_layer with row groups.
struct GroupedPlan {
  bool small;                // the small-output kernel
  int tile_m, tile_n;
  int64_t tiles_n;
  int64_t grid;              // workgroups of the launch
  bool a_direct, b_direct;   // operands read in place (else repacked)
  int64_t matrices;          // matrices B there are: the groups', or one for all
  size_t a_bytes, b_bytes;   // workspace of the repacked copies
  size_t total() const { return a_bytes + b_bytes; }
};

// A call of dense_gemm_tn.  The tiles of the groups' outputs (of the one
// output, without groups) form one sequence, `tiles_m * tiles_n` a group.
struct TnPlan {
  int64_t tile;              // tiles of tile x tile: 256 or 128
  int64_t tiles_m, tiles_n, groups;
  int64_t full_tasks;        // tiles computed whole
  int64_t split_tiles;       // tiles computed in K parts
  int64_t splits, steps;     // parts, and (without groups) K steps per part
  bool a_direct, b_direct;
  size_t a_bytes, b_bytes;
  size_t split_bytes;        // FP32 partial tiles
  size_t sums_bytes;         // the tasks' column sums of A (0: the tiles write them whole)
  size_t total() const { return a_bytes + b_bytes + split_bytes + sums_bytes; }
};

// The checks of dense_gemm_layer beyond dense_gemm_validate's, which they
// include.  *done: the call has nothing to compute.
dense_gemm_status layer_validate(int op, int64_t M, int64_t N, int64_t K, const void* A,
                                 int64_t lda, const void* B, int64_t ldb, const void* D,
                                 int64_t ldd, const dense_gemm_epilogue* e,
                                 const dense_gemm_groups* g, bool* done);

// The plan of a call of dense_gemm_layer without groups whose arguments passed
// layer_validate: plan_call's, or 128 x 128 tiles (plan[0] and plan[1]).
dense_gemm_status layer_plan(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                             int64_t lda, const void* B, int64_t ldb, int64_t cus, CallPlan* cp);

// The plan of a grouped call whose arguments passed layer_validate.
dense_gemm_status grouped_plan(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                               int64_t lda, const void* B, int64_t ldb, const dense_gemm_groups& g,
                               int64_t cus, GroupedPlan* out);

dense_gemm_status tn_validate(int fmt, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* B, int64_t ldb, const void* D, int64_t ldd,
                              const void* colsum, const dense_gemm_groups* g, bool* done);

dense_gemm_status tn_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                          const void* B, int64_t ldb, bool colsum, const dense_gemm_groups* g,
                          int64_t cus, TnPlan* out);

}  // namespace dg
