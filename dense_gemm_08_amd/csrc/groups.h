// groups.h -- rows sorted into groups (device side): the products of a
// mixture-of-experts layer, where the rows of one expert lie next to each
// other and each expert has a weight matrix of its own.
//
// Group g holds the rows ends[g - 1] .. ends[g] - 1 (ends[-1] = 0).  The ends
// live on the device: they come from the routing of the tokens, and the host
// need not wait for them.  So neither the number of output tiles nor their
// place is known at launch: each wave counts the groups' tiles once, one
// group per lane, and keeps the running counts in registers; finding a
// tile's group is then a compare and a ballot.  Every end is clamped to [0,
// rows] and raised to the ends before it, so whatever the array holds, no row
// outside [0, rows) is addressed, no row belongs to two groups, and the tiles
// number no more than the host allowed for.  (A.T @ B, whose tiles' places the
// host knows, reads a group's two ends alone, clamped but not raised: where
// ends decrease, groups may share rows.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

struct Groups {
  const int32_t* ends;  // count values, on the device
  int count;
  int rows;        // rows of the operands (rows at or past ends[count - 1] belong to no group)
  int64_t stride;  // elements between the groups' matrices (B, or D for A.T @ B)
};

__device__ __forceinline__ int clamp_end(const Groups& g, int end) {
  return min(max(end, 0), g.rows);
}

// ends[i], clamped, for an i that is the same in every lane: read through the
// constant address space, a scalar load, which waits for no vector-memory
// operation of the wave (the previous tile's stores keep draining).
__device__ __forceinline__ int group_end(const Groups& g, int i) {
  typedef const __attribute__((address_space(4))) int32_t* const_ptr;
  return clamp_end(g, ((const_ptr)(uintptr_t)g.ends)[i]);
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

// The largest x of this lane and those before it.
__device__ __forceinline__ int wave_max_scan(int x) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x = max(x, y);
  }
  return x;
}

// A tile's place: its group, its number within the group, the group's rows.
struct GroupTile {
  int group, tile;
  int beg, end;
};

// The running tile counts of the groups, tiles numbered group by group.  The
// first 64 HELD groups stay in registers (lane l of register c holds group 64
// c + l); those beyond are counted again from memory as tiles are looked up
// among them.  A workgroup's tile numbers only rise, so each lookup goes on
// from the 64 groups where the last one ended, and a launch walks the ends
// twice however many tiles it finds (2^14 groups of one row, N = K = 8: 4850
// us with a walk from the start for each tile, 496 so; 2^20 groups 33 ms).
template <int HELD>
struct GroupMap {
  int incl[HELD];  // tiles of this lane's group and all before it
  int end[HELD];   // the group's end
  int total;       // tiles there are
  // the groups past those held from which the next lookup goes on (64 c ..),
  // and the tiles and the end before them
  int at, at_tiles, at_end;

  // The tiles of this lane's group 64 c + lane, and its end; before: the end
  // of group 64 c - 1.
  __device__ __forceinline__ static int lane_tiles(const Groups& gr, int c, int before,
                                                   int tile_rows, int tiles_n, int* e) {
    const int lane = (int)threadIdx.x & 63, i = 64 * c + lane;
    *e = wave_max_scan(max(before, i < gr.count ? clamp_end(gr, gr.ends[i]) : 0));
    const int prev = __shfl_up(*e, 1);
    const int rows = *e - (lane > 0 ? prev : before);
    return (rows + tile_rows - 1) / tile_rows * tiles_n;
  }

  __device__ __forceinline__ void count(const Groups& gr, int tile_rows, int tiles_n) {
    total = 0;
    int before = 0;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      incl[c] = total;
      end[c] = before;
      if (64 * c < gr.count) {
        incl[c] += wave_scan(lane_tiles(gr, c, before, tile_rows, tiles_n, &end[c]));
        total = __builtin_amdgcn_readlane(incl[c], 63);
        before = __builtin_amdgcn_readlane(end[c], 63);
      }
    }
    at = HELD;
    at_tiles = total;
    at_end = before;
    for (int c = HELD; 64 * c < gr.count; ++c) {
      int e;
      total += __builtin_amdgcn_readlane(
          wave_scan(lane_tiles(gr, c, before, tile_rows, tiles_n, &e)), 63);
      before = __builtin_amdgcn_readlane(e, 63);
    }
  }

  // Among 64 groups' counts and ends, with the count and end before them.
  __device__ __forceinline__ static bool find_in(int incl, int end, int before, int beg, int c,
                                                 int tile, GroupTile* out) {
    const uint64_t past = __ballot(incl > tile);
    if (past == 0) return false;
    const int l = __builtin_ctzll(past);
    out->group = 64 * c + l;
    out->end = __builtin_amdgcn_readlane(end, l);
    out->beg = l > 0 ? __builtin_amdgcn_readlane(end, l - 1) : beg;
    out->tile = tile - (l > 0 ? __builtin_amdgcn_readlane(incl, l - 1) : before);
    return true;
  }

  // The place of tile `tile` (below total, and not below the last one asked
  // for).
  __device__ __forceinline__ void find(const Groups& gr, int tile, int tile_rows, int tiles_n,
                                       GroupTile* out) {
    int before = 0, beg = 0;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
      if (find_in(incl[c], end[c], before, beg, c, tile, out)) return;
      before = __builtin_amdgcn_readlane(incl[c], 63);
      beg = __builtin_amdgcn_readlane(end[c], 63);
    }
    for (; 64 * at < gr.count; ++at) {
      int e;
      const int n = at_tiles + wave_scan(lane_tiles(gr, at, at_end, tile_rows, tiles_n, &e));
      if (find_in(n, e, at_tiles, at_end, at, tile, out)) return;
      at_tiles = __builtin_amdgcn_readlane(n, 63);
      at_end = __builtin_amdgcn_readlane(e, 63);
    }
  }
};

}  // namespace dg
