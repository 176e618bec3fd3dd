// layer_host.h -- what the host sides of a layer's products share
// (layer.hip, grouped.hip, tn.hip): the call's arguments, and the kernel
// parameters made from them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense_gemm.h"
#include "gemm_small_kernel.h"
#include "layer_kernel.h"
#include "plan_layer.h"

namespace dg {

dense_gemm_status device_topology(int* cus, int* xcds);

// A copy of `count` matrices of rows x cols 16-bit elements, ld between their
// rows and stride between the matrices, into dense zero-padded ones at dst
// (null: none), whose leading dimension is repacked_ld(cols).
struct Repack {
  const void* src;
  void* dst;
  int64_t count, rows, cols, ld, stride;
};
inline int64_t repacked_ld(int64_t cols) { return (cols + 7) & ~(int64_t)7; }
// Enqueues one launch for both (none if neither is asked for): layer.hip.
void enqueue_repacks(const Repack& a, const Repack& b, hipStream_t stream);

inline dense_gemm_status launched() {
  return hipGetLastError() == hipSuccess ? DENSE_GEMM_OK : DENSE_GEMM_LAUNCH_FAILED;
}

inline Epilogue device_epilogue(const dense_gemm_epilogue* e) {
  Epilogue d = {};
  if (e == nullptr) return d;
  d.bias = (const uint16_t*)e->bias;
  d.bias_stride = e->bias != nullptr ? e->bias_stride : 0;
  d.res = (const uint16_t*)e->residual;
  d.z = (uint16_t*)e->preact;
  d.ldr = (int)e->ldr;
  d.ldz = (int)e->ldz;
  d.act = e->act;
  d.grad = e->grad;
  return d;
}

// One call's arguments, operands as the kernels read them (after repacks).
struct LayerCall {
  int64_t M, N, K;
  const uint16_t* A;
  int64_t lda;
  const uint16_t* B;
  int64_t ldb;
  uint16_t* D;
  int64_t ldd;
  const dense_gemm_epilogue* e;
  int cus, xcds;
  hipStream_t stream;
};

// Copies A (M x K) and the `count` matrices B (b_rows x b_cols) where a place
// for the copy is given, and makes the copies the call's operands.
inline void repack_operands(LayerCall& c, void* a_dst, int64_t count, int64_t b_rows,
                            int64_t b_cols, int64_t b_stride, void* b_dst) {
  enqueue_repacks({c.A, a_dst, 1, c.M, c.K, c.lda, 0},
                  {c.B, b_dst, count, b_rows, b_cols, c.ldb, b_stride}, c.stream);
  if (a_dst != nullptr) {
    c.A = (const uint16_t*)a_dst;
    c.lda = repacked_ld(c.K);
  }
  if (b_dst != nullptr) {
    c.B = (const uint16_t*)b_dst;
    c.ldb = repacked_ld(b_cols);
  }
}

inline void set_operands(LayerParams& p, const LayerCall& c) {
  p.A = c.A;
  p.B = c.B;
  p.D = c.D;
  p.M = (int)c.M;
  p.N = (int)c.N;
  p.K = (int)c.K;
  p.lda = (int)c.lda;
  p.ldb = (int)c.ldb;
  p.ldd = (int)c.ldd;
  p.num_xcds = c.xcds;
}

inline SmallLayerParams small_params(const LayerCall& c) {
  SmallLayerParams p = {};
  p.A = c.A;
  p.B = c.B;
  p.D = c.D;
  p.M = (int)c.M;
  p.N = (int)c.N;
  p.K = (int)c.K;
  p.K8 = (int)((c.K + 7) & ~(int64_t)7);
  p.N8 = (int)((c.N + 1) & ~(int64_t)1);  // (columns of B that may be read: whole words)
  p.lda = (int)c.lda;
  p.ldb = (int)c.ldb;
  p.ldd = (int)c.ldd;
  p.num_xcds = c.xcds;
  p.d_vec = 1;
  p.e = device_epilogue(c.e);
  return p;
}

// grouped.hip: a call with row groups.
template <typename T, int LAYOUT>
dense_gemm_status run_grouped(LayerCall c, const dense_gemm_groups& groups, void* ws,
                              size_t ws_bytes);

}  // namespace dg
