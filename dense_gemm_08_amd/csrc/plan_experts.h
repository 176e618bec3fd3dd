// plan_experts.h -- host-side checks and plans of what stands around an expert
// layer's products, and of the int8 products (plain C++, no device code).
// Implemented in plan_experts.cpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "plan_layer.h"

namespace dg {

// ---- routing ----

constexpr int ROUTE_MOST_EXPERTS = 1024;
constexpr int ROUTE_MOST_K = 64;
constexpr int ROUTE_MOST_GROUPS = 64;
constexpr int ROUTE_THREADS = 1024;
// Choices (tokens times k): the kernels look a block's tokens past the end in 32
// bits.
constexpr int64_t kRouteMostRows = kMaxDim - (1 << 20);

struct RoutePlan {
  int64_t chunks;  // chunks of 64 tokens per block
  int64_t blocks;  // 1: one launch; more: a second one makes the dispatch
  size_t bytes;    // workspace
};

// Checks of dense_gemm_route; without tokens it still writes the ends.
dense_gemm_status route_validate(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                 int64_t ldl, const dense_gemm_routing* r, const void* weights,
                                 const void* experts, const void* places, const void* ends,
                                 const void* tokens);
dense_gemm_status route_grad_validate(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                      int64_t ldl, const dense_gemm_routing* r, const void* experts,
                                      const void* dweights, const void* dlogits, int64_t ldd,
                                      bool* done);
RoutePlan route_plan(int64_t T, int64_t E);

// ---- rows ----

// Lanes that share a row of `cols` elements, of `rows` rows: 16, 64, 256 or
// 1024.
int row_lanes(int64_t rows, int64_t cols, int64_t cus);

dense_gemm_status quantize_validate(int fmt, int64_t R, int64_t K, const void* X, int64_t ldx,
                                    int64_t x_rows, const void* rows, const void* Q, int64_t ldq,
                                    const void* S, bool* done);
dense_gemm_status combine_validate(int fmt, int64_t T, int64_t N, int64_t k, const void* H, int64_t ldh,
                                   int64_t h_rows, const void* places, const void* weights,
                                   const void* residual, int64_t ldr, const void* Y, int64_t ldy,
                                   bool* done);
dense_gemm_status combine_grad_validate(int fmt, int64_t T, int64_t N, int64_t k, const void* DY,
                                        int64_t lddy, const void* H, int64_t ldh, int64_t h_rows,
                                        const void* places, const void* weights, const void* DH,
                                        int64_t lddh, const void* dweights, bool* done);

// ---- int8 products ----

// The largest K whose sums fit 32 bits whatever the values: K 2^14 < 2^31.
constexpr int64_t I8_MOST_K = (1 << 17) - 1;

// The kernels take rows of K bytes as rows of 16-bit pairs; a call's plan is the
// one of a 16-bit product with half the K, and the copies it needs are by
// bytes.
dense_gemm_status i8_validate(int fmt, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* SA, const void* B, int64_t ldb, const void* SB,
                              const void* D, int64_t ldd, const dense_gemm_epilogue* e,
                              const dense_gemm_groups* g, int64_t sb_stride, bool* done);
dense_gemm_status i8_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                          int64_t ldb, int64_t cus, CallPlan* cp);
dense_gemm_status i8_grouped_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                  const void* B, int64_t ldb, const dense_gemm_groups& g, int64_t cus,
                                  GroupedPlan* out);

}  // namespace dg
