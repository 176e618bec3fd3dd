// column_sums.h -- the last step of the column sums of A that accompany D =
// A.T @ B on the MI355X (gfx950): layer_gemm_kernel<..., SUMS> leaves FP32 sums over
// shares of K, here they are added in a fixed order and rounded once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"

namespace dg {

struct ColumnSumsParams {
  const float* ws;  // two rows of TM sums per task
  uint16_t* out;    // groups x M
  int M, groups;
  int tiles_m, tiles_n, group_m;
  // tasks below full_tasks are whole tiles, then come `splits` parts of each
  // of the last `tiles` tiles (layer_kernel.h)
  int full_tasks, splits, tiles;
};

// Block `block` of M / 16 x groups adds 16 columns of one group: 16 lanes hold
// the columns of a row of sums, and the block's rows of lanes take every
// CS_LANES-th of the rows of sums that the column's tiles left, four loads in
// flight at a time; their sums are then added through LDS in order.  Bound by
// the latency of those loads.  (Where the product has a second kernel
// already, split_reduce.h, these blocks join its launch: 512 x 640 x 20011
// 32 -> 31 us.)
constexpr int CS_COLS = 16;
inline int64_t column_sums_blocks(int64_t M, int64_t groups) {
  return groups * ((M + CS_COLS - 1) / CS_COLS);
}
template <typename T, int TM, int RT>
__device__ __forceinline__ void column_sums_block(const ColumnSumsParams& p, int block) {
  constexpr int CS_LANES = RT / CS_COLS;
  __shared__ float part[CS_LANES][CS_COLS];
  const int per_group = (p.M + CS_COLS - 1) / CS_COLS;
  const int g = block / per_group;
  const int c = (int)threadIdx.x % CS_COLS, r = (int)threadIdx.x / CS_COLS;
  const int m = (block - g * per_group) * CS_COLS + c;
  const int tm = m / TM;
  // tile (tm, tn) of the group in the grouped order (tile_sched.h)
  const int first_m = tm / p.group_m * p.group_m;
  const int gsize = min(p.group_m, p.tiles_m - first_m);
  const int tile0 = g * p.tiles_m * p.tiles_n + first_m * p.tiles_n + tm - first_m;
  float s = 0.0f;
  if (m < p.M) {
    const int rows = p.tiles_n * 2 * p.splits;
    constexpr int U = 4;
    for (int i0 = r; i0 < rows; i0 += U * CS_LANES) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * CS_LANES;
        const int tn = i / (2 * p.splits), k = i % (2 * p.splits) / 2;
        const int tile = tile0 + tn * gsize;
        const bool whole = tile < p.full_tasks;
        const int64_t task = whole ? tile : (int64_t)k * p.tiles + tile;
        x[u] = i < rows && !(whole && k > 0) ? p.ws[(task * 2 + i % 2) * TM + m % TM] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) s += x[u];
    }
  }
  part[r][c] = s;
  __syncthreads();
  if (r == 0 && m < p.M) {
    s = part[0][c];
#pragma unroll
    for (int i = 1; i < CS_LANES; ++i) s += part[i][c];
    p.out[(int64_t)g * p.M + m] = (uint16_t)pack2<T>(s, 0.0f);
  }
}

// The sums alone, in up to CS_MAX_GRID workgroups (a launch holds fewer than
// 2^32 threads, many groups can have more blocks than that).
constexpr int CS_THREADS = 256;
constexpr int64_t CS_MAX_GRID = 1 << 16;
template <typename T, int TM>
__global__ __launch_bounds__(CS_THREADS) void column_sums(ColumnSumsParams p, int blocks) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    column_sums_block<T, TM, CS_THREADS>(p, (int)b);
    __syncthreads();
  }
}

}  // namespace dg
