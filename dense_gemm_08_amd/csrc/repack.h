// repack.h -- copies of operands that the layer products' LDS-DMA loads cannot
// read in place (plan_layer.cpp: direct; rows of an odd length or at an odd
// distance, mostly) into dense, zero-padded matrices, on the MI355X (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"
#include "epilogue.h"

namespace dg {

constexpr int64_t REPACK_GROUPS_MAX_BLOCKS = 1 << 16;

// A copy of `count` matrices of rows x cols 16-bit elements (any leading
// dimension and distance, 2-byte alignment) into dense, 16-byte aligned ones
// of rows x dcols (dcols = cols rounded up to 8), zero-filling the columns
// past cols: what the kernels' 16-byte loads need.
struct RepackJob {
  const uint16_t* src;
  uint16_t* dst;
  int64_t count, rows, cols, ld, stride, dcols;
  int64_t blocks;  // workgroups of the launch that do this job
  int lanes;       // lanes per row, a power of two up to 256
};

// Two such copies (one may have no blocks).  Bound by memory: a lane moves 8
// elements at a time with one load of any alignment and one aligned store;
// a workgroup takes 256 / lanes rows at a time and strides over the rest.
// 1001 x 2051 and 777 x 2051 elements: 3 us together, 7 us each when a lane
// loaded element by element.
[[maybe_unused]] static __global__ __launch_bounds__(256) void repack_groups(RepackJob a,
                                                                             RepackJob b) {
  const bool first = blockIdx.x < a.blocks;
  const RepackJob& j = first ? a : b;
  const int64_t block = first ? blockIdx.x : blockIdx.x - a.blocks;
  const int shift = __builtin_ctz(j.lanes), lane = (int)threadIdx.x & (j.lanes - 1);
  const int per = 256 >> shift;
  const int64_t total = j.count * j.rows;
  for (int64_t r = block * per + ((int)threadIdx.x >> shift); r < total; r += j.blocks * per) {
    const int64_t g = j.count > 1 ? r / j.rows : 0;
    const uint16_t* src = j.src + g * j.stride + (r - g * j.rows) * j.ld;
    for (int64_t c = lane * 8; c < j.dcols; c += j.lanes * 8) {
      uint32_t w[4];
      load_row<4>(src, (int)c, (int)j.cols, w);
      *(u32x4*)(j.dst + r * j.dcols + c) = (u32x4){w[0], w[1], w[2], w[3]};
    }
  }
}

}  // namespace dg
