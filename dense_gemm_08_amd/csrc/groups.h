// groups.h -- rows sorted into groups (device side): the products of a
// mixture-of-experts layer, where the rows of one expert lie next to each
// other and each expert has a weight matrix of its own.
//
// Group g holds the rows ends[g - 1] .. ends[g] - 1 (ends[-1] = 0).  The ends
// live on the device: they come from the routing of the tokens, and the host
// need not wait for them.  So neither the number of output tiles nor their
// place is known at launch; a workgroup finds the group of its next tile by
// walking the groups (its tiles come in rising order, so it only ever walks
// forwards).  Every end is clamped to [0, rows], and a group whose end lies
// before its beginning is empty: whatever the array holds, no row outside
// [0, rows) is addressed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tile_sched.h"

namespace dg {

struct Groups {
  const int32_t* ends;  // count values, on the device
  int count;
  int rows;        // rows of the operands (rows at or past ends[count - 1] belong to no group)
  int64_t stride;  // elements between the groups' matrices (B, or D for A.T @ B)
};

// ends[i], clamped.  Read through the constant address space: i is the same
// in every lane, so this is a scalar load, which waits for no vector-memory
// operation of the wave (the previous tile's stores keep draining).
__device__ __forceinline__ int group_end(const Groups& g, int i) {
  typedef const __attribute__((address_space(4))) int32_t* const_ptr;
  const int v = ((const_ptr)(uintptr_t)g.ends)[i];
  return min(max(v, 0), g.rows);
}

// The group that holds an output tile, tiles numbered group by group.
struct GroupWalk {
  int g;         // current group
  int first;     // number of its first tile
  int beg, end;  // its rows
  __device__ __forceinline__ void start(const Groups& gr) {
    g = 0;
    first = 0;
    beg = 0;
    end = group_end(gr, 0);
  }
  // Walks to the group of tile `task` (not before the current group); false
  // if there is no such tile.
  __device__ __forceinline__ bool find(const Groups& gr, int task, int tile_rows, int tiles_n) {
    for (;;) {
      const int here = end > beg ? (end - beg + tile_rows - 1) / tile_rows * tiles_n : 0;
      if (task < first + here) return true;
      first += here;
      if (++g >= gr.count) return false;
      beg = end;
      end = group_end(gr, g);
    }
  }
};

// The tile of a workgroup when the launch holds one workgroup per possible
// tile: workgroup b of the `total` that have a tile takes tile
// xcd_slot(b, total) (tile_sched.h), so that neighbouring tiles run on one
// XCD however many there are.  All lanes of a wave search together, 64
// groups at a time.
struct GroupTile {
  int group, tile;  // the group, and the tile's number within it
  int beg, end;     // the group's rows
};

__device__ __forceinline__ int lane_tiles(const Groups& gr, int i, int tile_rows, int tiles_n,
                                          int* beg, int* end) {
  const bool live = i < gr.count;
  *end = live ? min(max(gr.ends[i], 0), gr.rows) : 0;
  *beg = live && i > 0 ? min(max(gr.ends[i - 1], 0), gr.rows) : 0;
  return *end > *beg ? (*end - *beg + tile_rows - 1) / tile_rows * tiles_n : 0;
}

// The sum of x over this lane and those before it.
__device__ __forceinline__ int wave_scan(int x) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ bool find_tile(const Groups& gr, int b, int num_xcds, int tile_rows,
                                          int tiles_n, GroupTile* out) {
  const int lane = (int)threadIdx.x & 63;
  int total = 0, beg, end, mine, incl;
  for (int c = 0; c < gr.count; c += 64) {
    mine = lane_tiles(gr, c + lane, tile_rows, tiles_n, &beg, &end);
    incl = wave_scan(mine);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  if (b >= total) return false;
  const int slot = xcd_slot(b, total, num_xcds);
  int first = 0;
  for (int c = 0; c < gr.count; c += 64) {
    if (gr.count > 64) {  // (else the values of the only pass above still stand)
      mine = lane_tiles(gr, c + lane, tile_rows, tiles_n, &beg, &end);
      incl = wave_scan(mine);
    }
    const uint64_t past = __ballot(first + incl > slot);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      out->group = c + l;
      out->tile = slot - first - __builtin_amdgcn_readlane(incl - mine, l);
      out->beg = __builtin_amdgcn_readlane(beg, l);
      out->end = __builtin_amdgcn_readlane(end, l);
      return true;
    }
    first += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

}  // namespace dg
