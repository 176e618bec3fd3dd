// i8.hip -- a layer's products with int8 operands and a scale per row of each
// (dense_gemm_i8, include/dense_gemm.h) on the MI355X (gfx950).  Host side: the
// plans (plan_experts.cpp), the launches and the C ABI entry points.  The
// kernels are layer_gemm_kernel with int8 operands (layer_kernel.h, i8.h) and
// gemm_small_i8 (i8_small_kernel.h).
#include "i8_small_kernel.h"
#include "layer_host.h"
#include "plan_experts.h"

namespace dg {

namespace {

struct I8Call {
  int64_t M, N, K;
  const int8_t* A;
  int64_t lda;
  const int8_t* B;
  int64_t ldb;
  uint16_t* D;
  int64_t ldd;
  I8Scales s;
  const dense_gemm_epilogue* e;
  int cus, xcds;
  hipStream_t stream;
};

// Copies A and the `count` matrices B where a place for the copy is given, and
// makes the copies the call's operands.
void repack(I8Call& c, void* a_dst, int64_t count, int64_t b_stride, void* b_dst) {
  const int64_t dcols = (c.K + 15) & ~(int64_t)15;
  I8RepackJob job[2] = {};
  int64_t grid = 0;
  auto add = [&](I8RepackJob& j, const int8_t* src, void* dst, int64_t n, int64_t rows, int64_t ld,
                 int64_t stride) {
    if (dst == nullptr) return;
    j = {src, (int8_t*)dst, n, rows, c.K, ld, stride, dcols, 0, 1};
    while (j.lanes < 256 && j.lanes * 16 < dcols) j.lanes *= 2;
    const int64_t per = 256 / j.lanes;
    j.blocks = (n * rows + per - 1) / per;
    if (j.blocks > 1 << 16) j.blocks = 1 << 16;
    grid += j.blocks;
  };
  add(job[0], c.A, a_dst, 1, c.M, c.lda, 0);
  add(job[1], c.B, b_dst, count, c.N, c.ldb, b_stride);
  if (grid > 0)
    hipLaunchKernelGGL(repack_i8, dim3((unsigned)grid), dim3(256), 0, c.stream, job[0], job[1]);
  if (a_dst != nullptr) {
    c.A = (const int8_t*)a_dst;
    c.lda = dcols;
  }
  if (b_dst != nullptr) {
    c.B = (const int8_t*)b_dst;
    c.ldb = dcols;
  }
}

SmallI8Params small_params(const I8Call& c) {
  SmallI8Params p = {};
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
  p.e = device_epilogue(c.e);
  p.s = c.s;
  return p;
}

// (rows of K bytes as rows of pairs)
LayerI8Params tiled_params(const I8Call& c) {
  LayerI8Params p = {};
  p.A = (const uint16_t*)c.A;
  p.B = (const uint16_t*)c.B;
  p.D = c.D;
  p.M = (int)c.M;
  p.N = (int)c.N;
  p.K = (int)(2 * ((c.K + 3) / 4));
  p.lda = (int)(c.lda / 2);
  p.ldb = (int)(c.ldb / 2);
  p.ldd = (int)c.ldd;
  p.num_xcds = c.xcds;
  p.e = device_epilogue(c.e);
  p.s = c.s;
  return p;
}

template <typename O, int TN, int TM>
dense_gemm_status enqueue_tiled(const I8Call& c, const CallPlan& cp, void* parts) {
  LayerI8Params p = tiled_params(c);
  p.tiles_m = (int)cp.plan[3];
  p.tiles_n = (int)cp.plan[4];
  p.group_m = (int)cp.plan[6];
  p.full_tasks = (int)cp.full_tasks;
  p.tiles = (int)cp.split_tiles;
  p.splits = (int)cp.plan[8];
  p.split_steps = (int)cp.plan[9];
  p.num_tasks = (int)(cp.full_tasks + cp.split_tiles * cp.plan[8]);
  p.ws = (float*)parts;
  const int slots = c.cus * (int)resident(TM, TN);
  const dim3 grid((unsigned)(p.num_tasks < slots ? p.num_tasks : slots)), block(THREADS);
  if (p.splits > 1 || (resident(TM, TN) > 1 && p.num_tasks <= c.cus)) {
    hipLaunchKernelGGL((layer_gemm_kernel<I8<O>, NT, true, TN, TM, false>), grid, block, 0, c.stream, p);
    if (p.splits == 1) return launched();
    const I8ReduceParams r = {(const int32_t*)parts, p.D, p.M, p.N, p.ldd, p.tiles_m, p.tiles_n,
                              p.group_m, p.full_tasks, p.splits, p.tiles, p.e, p.s};
    constexpr int per_tile = TM * TN / 8 / I8_REDUCE_THREADS;
    hipLaunchKernelGGL((split_reduce_i8<O, TN, TM>), dim3((unsigned)(p.tiles * per_tile)),
                       dim3(I8_REDUCE_THREADS), 0, c.stream, r);
  } else {
    hipLaunchKernelGGL((layer_gemm_kernel<I8<O>, NT, false, TN, TM, false>), grid, block, 0, c.stream, p);
  }
  return launched();
}

template <typename O>
dense_gemm_status run(I8Call c, void* ws, size_t ws_bytes) {
  CallPlan cp;
  const dense_gemm_status st = i8_plan(c.M, c.N, c.K, c.A, c.lda, c.B, c.ldb, c.cus, &cp);
  if (st != DENSE_GEMM_OK) return st;
  if (cp.total() > 0) {
    if (ws == nullptr || ws_bytes < cp.total()) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)ws & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  char* at = (char*)ws;
  repack(c, cp.a_direct ? nullptr : at, 1, 0, cp.b_direct ? nullptr : at + cp.a_bytes);
  at += cp.a_bytes + cp.b_bytes;
  if (cp.small()) {
    SmallI8Params p = small_params(c);
    p.tiles_m = (int)cp.plan[3];
    p.tiles_n = (int)cp.plan[4];
    const dim3 grid((unsigned)(cp.plan[3] * cp.plan[4])), block(SMALL_THREADS);
    if (cp.plan[0] != 2 * SMALL_TILE)
      hipLaunchKernelGGL((gemm_small_i8<O, 1, 1, false>), grid, block, 0, c.stream, p);
    else if (cp.plan[1] == 2 * SMALL_TILE)
      hipLaunchKernelGGL((gemm_small_i8<O, 2, 2, false>), grid, block, 0, c.stream, p);
    else
      hipLaunchKernelGGL((gemm_small_i8<O, 2, 1, false>), grid, block, 0, c.stream, p);
    return launched();
  }
  const bool short_tiles = cp.plan[0] == BM / 2, narrow = cp.plan[1] == BN / 2;
  if (short_tiles)
    return narrow ? enqueue_tiled<O, BN / 2, BM / 2>(c, cp, at) : enqueue_tiled<O, BN, BM / 2>(c, cp, at);
  return narrow ? enqueue_tiled<O, BN / 2, BM>(c, cp, at) : enqueue_tiled<O, BN, BM>(c, cp, at);
}

template <typename O>
dense_gemm_status run_grouped(I8Call c, const dense_gemm_groups& groups, void* ws, size_t ws_bytes) {
  GroupedPlan gp;
  const dense_gemm_status st = i8_grouped_plan(c.M, c.N, c.K, c.A, c.lda, c.B, c.ldb, groups, c.cus, &gp);
  if (st != DENSE_GEMM_OK) return st;
  if (gp.total() > 0) {
    if (ws == nullptr || ws_bytes < gp.total()) return DENSE_GEMM_WORKSPACE_TOO_SMALL;
    if (((uintptr_t)ws & 255) != 0) return DENSE_GEMM_MISALIGNED;
  }
  Groups g = {(const int32_t*)groups.ends, (int)groups.count, (int)c.M, groups.stride};
  repack(c, gp.a_direct ? nullptr : ws, gp.matrices, g.stride,
         gp.b_direct ? nullptr : (char*)ws + gp.a_bytes);
  if (!gp.b_direct && gp.matrices > 1) g.stride = c.N * c.ldb;
  const dim3 grid((unsigned)gp.grid);
  if (gp.small) {
    SmallI8Params p = small_params(c);
    p.tiles_n = (int)gp.tiles_n;
    p.g = g;
    hipLaunchKernelGGL((gemm_small_i8<O, 1, 1, true>), grid, dim3(SMALL_THREADS), 0, c.stream, p);
    return launched();
  }
  LayerI8Params p = tiled_params(c);
  p.tiles_n = (int)gp.tiles_n;
  p.group_m = choose_group_m(kMaxDim);
  p.g = g;
  p.g.stride = g.stride / 2;
  if (gp.tile_n == BN / 2)
    hipLaunchKernelGGL((layer_gemm_kernel<I8<O>, NT, false, BN / 2, BM / 2, true>), grid, dim3(THREADS), 0,
                       c.stream, p);
  else
    hipLaunchKernelGGL((layer_gemm_kernel<I8<O>, NT, false, BN, BM, true>), grid, dim3(THREADS), 0,
                       c.stream, p);
  return launched();
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

dense_gemm_status dense_gemm_i8(int fmt, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                const void* SA, const void* B, int64_t ldb, const void* SB,
                                int64_t sb_stride, void* D, int64_t ldd,
                                const dense_gemm_epilogue* epilogue, const dense_gemm_groups* groups,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  bool done;
  dense_gemm_status st = i8_validate(fmt, M, N, K, A, lda, SA, B, ldb, SB, D, ldd, epilogue, groups,
                                     sb_stride, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  I8Call c = {M, N, K, (const int8_t*)A, lda, (const int8_t*)B, ldb, (uint16_t*)D, ldd,
              {(const float*)SA, (const float*)SB, groups != nullptr ? sb_stride : 0},
              epilogue, 0, 1, stream};
  st = device_topology(&c.cus, &c.xcds);
  if (st != DENSE_GEMM_OK) return st;
  if (groups != nullptr)
    return fmt == DENSE_GEMM_BF16 ? run_grouped<__bf16>(c, *groups, workspace, workspace_bytes)
                                  : run_grouped<_Float16>(c, *groups, workspace, workspace_bytes);
  return fmt == DENSE_GEMM_BF16 ? run<__bf16>(c, workspace, workspace_bytes)
                                : run<_Float16>(c, workspace, workspace_bytes);
}

dense_gemm_status dense_gemm_i8_workspace_size(int64_t M, int64_t N, int64_t K, const void* A,
                                               int64_t lda, const void* B, int64_t ldb,
                                               const dense_gemm_groups* groups, int64_t num_cus,
                                               size_t* bytes) {
  if (bytes == nullptr || num_cus < 0) return DENSE_GEMM_BAD_ARG;
  const void* any = (const void*)(uintptr_t)16;
  dense_gemm_groups g = {any, 0, 0};
  if (groups != nullptr) {
    g.count = groups->count;
    g.stride = groups->stride;
  }
  bool done;
  dense_gemm_status st = i8_validate(DENSE_GEMM_BF16, M, N, K, A, lda, any, B, ldb, any, any, N, nullptr,
                                     groups != nullptr ? &g : nullptr, 0, &done);
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
    st = i8_grouped_plan(M, N, K, A, lda, B, ldb, g, cus, &gp);
    if (st == DENSE_GEMM_OK) *bytes = gp.total();
    return st;
  }
  CallPlan cp;
  st = i8_plan(M, N, K, A, lda, B, ldb, cus, &cp);
  if (st == DENSE_GEMM_OK) *bytes = cp.total();
  return st;
}

}  // extern "C"
