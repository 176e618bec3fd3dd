// gemm_kernel.h -- the FP16/BF16 tiled GEMM kernel for the MI355X (gfx950):
// the persistent GEMM kernel (the split-K reduction is in split_reduce.h,
// the operand repack in repack.h).
//
// Kernel structure (one persistent workgroup per CU):
//   * a persistent loop over output tiles in the grouped, XCD-aware order of
//     tile_sched.h ("TIRx GEMM on Blackwell", V6: persistent CTAs pulling
//     tiles; TileFoundry schedule tutorial, sections 2-3: persistent CTAs and
//     the grouped traversal);
//   * per K step, 16-byte LDS-DMA loads of the A and B tiles into LDS rings
//     (three slots for one operand, two for the other: all 160 KiB) while
//     the previous stage feeds the matrix cores ("TIRx GEMM on Blackwell",
//     V5: shared-memory stages so loading the next K tile overlaps the MMA
//     of the current one);
//   * an XOR swizzle of 16-byte chunks inside each LDS row, so both the
//     row-wise tile writes and the column-wise MFMA fragment reads spread over
//     all banks (the role of the 128-byte swizzle in the TIRx and TileFoundry
//     shared-memory layouts);
//   * v_mfma_f32_16x16x32_{f16,bf16} with FP32 accumulators; four waves each
//     own a 128 x 128 quarter of a 256 x 256 tile (128 x 64 of a 256 x 128
//     tile for narrow A @ B.T outputs; 64 rows of a 128-row tile where M <=
//     128) and read the shared A and B stages
//     ("TIRx GEMM on Blackwell", V8/V9: larger tiles and several consumers
//     reusing one staged operand tile);
//   * an epilogue that rounds to the output type, stages each wave's rows in
//     LDS and writes whole 16-byte row chunks (TileFoundry tutorial, section 5:
//     the output tile is staged in shared memory before the store);
//   * ragged M, N and K handled by masking: out-of-range loads read zeros
//     through the buffer descriptor's range check, out-of-range stores are
//     skipped (the pages' shapes all divide the tiles; this is our reading);
//   * split-K for the last, partial wave of tiles (the parts' FP32 tiles
//     summed by split_reduce.h), and a repack of operands the 16-byte loads
//     cannot read in place (chosen by the host side, dense_gemm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cdna_ops.h"
#include "epilogue.h"
#include "groups.h"
#include "tile_config.h"
#include "tile_sched.h"

namespace dg {

// ---- tile configuration (Layout, BM, BN, BK, WAVES, THREADS: tile_config.h)
constexpr int MK = 32;               // K depth of one MFMA (16 x 16 x 32)
constexpr int SUB = BK / MK;         // MFMA k-substeps per stage
// Tile rows TM: 256 (BM), or 128 for products with M <= 128 (half the
// MFMA work of a 256-row tile that would be half padding).  A wave tile is
// TM / 2 rows (MI 16-row MFMA blocks); the A tile of a stage is TM rows of
// 128 B, loaded in TM / 32 16-byte loads per thread.
template <int TM>
constexpr int wave_rows() { return TM / 2; }
template <int TM>
constexpr int a_loads() { return TM * BK * 2 / (THREADS * 16); }
// MFMA pairs of the last substep issued before its barrier: the reads of
// that substep's fragments (issued during the previous substep) complete
// meanwhile, so the barrier's LDS wait costs nothing
constexpr int BAR_PAIR = 2;

static_assert(BK == 64 && BM == 256 && BN == 256, "swizzles below assume these sizes");
static_assert(SUB == 2, "the ring schedule below has two substeps per stage");

struct Params {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* D;
  int M, N, K;
  int lda, ldb, ldd;
  int tiles_m, tiles_n, group_m, num_tasks, num_xcds;
  int d_vec;  // D rows are 16-byte aligned (16-byte stores allowed)
  // split-K (the SPLIT kernels): tasks below full_tasks are whole tiles;
  // the rest are (tile, part) pairs over the last `tiles` tiles of the
  // order.  Task full_tasks + u is part u / tiles of tile full_tasks +
  // u % tiles; the part covers K steps [part * split_steps, min(nk, (part +
  // 1) * split_steps)) and writes its FP32 partial tile (row-major TM x TN,
  // TM and TN the tile's rows and width) to ws at index part * tiles + u %
  // tiles
  int full_tasks, splits, split_steps, tiles;
  float* ws;
};

// What the products of a layer (layer.hip) add: the epilogue's operands
// (epilogue.h), the row groups (groups.h) and the column sums of A (SUMS):
// each task leaves its two wave columns' FP32 sums of its TM columns at
// colsum_ws + task * 2 TM (added up by column_sums, column_sums.h).
struct LayerParams : Params {
  Epilogue e;
  Groups g;
  float* colsum_ws;
};

// Stages loaded ahead of the one in use.  Two, with rings of three slots for
// one operand and two for the other, fill the LDS for 256-wide tiles.  The
// 128 x 128 tiles of the layer products are 80 KiB that way:
//   * many tiles run two workgroups per CU, so that one computes while the
//     other waits for its first tiles or writes its last ones;
//   * at most one tile or part per CU (the SPLIT kernels) runs four stages
//     ahead instead, in 144 KiB, to cover the load latency alone.
template <int LAYOUT, bool SPLIT, int TN, int TM, bool EPI, bool GROUP>
constexpr bool pair_tile() {
  return TM == BM / 2 && TN == BN / 2 && (EPI || GROUP || LAYOUT == TA);
}
template <int LAYOUT, bool SPLIT, int TN, int TM, bool EPI, bool GROUP>
constexpr int stages_ahead() {
  return pair_tile<LAYOUT, SPLIT, TN, TM, EPI, GROUP>() && SPLIT ? 4 : 2;
}
template <int LAYOUT, bool SPLIT, int TN, int TM, bool EPI, bool GROUP>
constexpr int per_cu() {
  return pair_tile<LAYOUT, SPLIT, TN, TM, EPI, GROUP>() && !SPLIT ? 2 : 1;
}

template <int MA, int NB>
struct Frags {
  u32x4 a[MA];
  u32x4 b[NB];
};

// Tile width TN: 256 (four 128 x 128 wave tiles), or for A @ B.T 128 (four
// 128 x 64 wave tiles): for outputs at most 128 wide (half the work of a
// half-padded 256-wide tile), and for twice the tiles where 256-wide ones
// would leave half the CUs idle, at more operand traffic per FLOP.  Tile
// rows TM: 256, or 128 where M <= 128 (four 64-row wave tiles).
//
// Three further parameters serve the products of a layer:
//   LAYOUT TA  D = A.T @ B with A K x M and B K x N, both row-major: both
//              tiles are 64 k rows of 512 B, read with transposing LDS reads;
//   EPI        bias, activation, residual or activation gradient applied to
//              the accumulators before the one rounding (epilogue.h);
//   GROUP      rows sorted into groups (groups.h): for A @ B.T and A @ B a
//              matrix B per group of rows of A and D; for A.T @ B a sum over
//              each group's rows, and an output matrix per group;
//   SUMS       (TA) also the sums of A's columns over k.
template <typename T, int LAYOUT, bool SPLIT, int TN, int TM, bool EPI = false, bool GROUP = false,
          bool SUMS = false>
__global__ __launch_bounds__(THREADS, (per_cu<LAYOUT, SPLIT, TN, TM, EPI, GROUP>())) void gemm_kernel(
    std::conditional_t<EPI || GROUP || LAYOUT == TA, LayerParams, Params> p) {
  static_assert(TN == BN || TN == BN / 2, "tile widths 256 and 128");
  static_assert(TM == BM || TM == BM / 2, "tile rows 256 or 128");
  static_assert(LAYOUT != TA || TM == TN, "A.T @ B takes square tiles");
  static_assert(!(EPI && LAYOUT == TA), "no epilogue on A.T @ B");
  static_assert(!SUMS || LAYOUT == TA, "column sums of A where its rows are k");
  static_assert(!(GROUP && SPLIT && LAYOUT != TA), "row groups are not split in K");
  constexpr int WTM = wave_rows<TM>();             // wave tile rows
  constexpr int MI = WTM / 16;                     // 16 x 16 blocks per wave, M direction
  constexpr int A_BYTES = TM * BK * 2;             // bytes of an A tile (TM rows x 128 B)
  constexpr int DMA_PER_OPERAND = a_loads<TM>();   // 16-byte loads per thread (A)
  constexpr int WTN = TN / 2;                      // wave tile columns
  constexpr int NI = WTN / 16;                     // 16 x 16 blocks per wave, N direction
  constexpr int PAIRS = MI * NI / 2;               // MFMA pairs per substep
  constexpr int B_TILE = TN * BK * 2;              // bytes of a B tile
  constexpr int DMA_B = B_TILE / (THREADS * 16);   // 16-byte loads per thread (B)
  // The operand with the three-slot ring, whose loads are issued a substep
  // earlier (0 = A, 1 = B): B for A @ B, whose row-major tile (64 rows of
  // 512 B, far apart in memory) is the costlier one to load (measured: 1.4%
  // faster than A there); A for A @ B.T (the two are alike).
  constexpr int EARLY = LAYOUT == NT ? 0 : 1;
  constexpr bool ROWS = GROUP && LAYOUT != TA;  // groups of rows of A and D
  constexpr int DMA_E = EARLY == 0 ? DMA_PER_OPERAND : DMA_B;   // loads of the early tile
  constexpr int DMA_L = EARLY == 0 ? DMA_B : DMA_PER_OPERAND;   // and of the other
  constexpr int E_BYTES = EARLY == 0 ? A_BYTES : B_TILE;
  constexpr int L_BYTES = EARLY == 0 ? B_TILE : A_BYTES;
  constexpr int AHEAD = stages_ahead<LAYOUT, SPLIT, TN, TM, EPI, GROUP>();
  constexpr int RING2 = (AHEAD + 1) * E_BYTES;       // the other ring follows the early one
  constexpr int LDS_BYTES = RING2 + AHEAD * L_BYTES;   // all 160 KiB for 256-wide tiles
  using Frags = dg::Frags<MI, NI>;
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
  const uint32_t lds0 = lds_addr(smem);

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1;  // wave tile row (0..1)
  const int wn = wave & 1;   // wave tile column (0..1)

  // Where all tasks are alike, the layer products deal each XCD one run of
  // them, an even share, which its workgroups take in turn: the tasks of a
  // last, partial round then fall on all XCDs, a few CUs each (48 groups,
  // 5003 rows, 63 -> 53 us; A.T @ B 5120 x 8192 x 8192, 2.5 rounds, 551 ->
  // 533).  Else the tasks are dealt round by round, so that a round's tiles
  // are neighbours over all XCDs: groups of different K would leave the XCDs
  // with different work (16 groups' A.T @ B 508 us, 1254 in runs), and 16
  // groups of 1024 rows take 509 us, 523 in runs.
  constexpr bool SHARES = !SPLIT && (GROUP ? ROWS && TM == BM / 2 : EPI || LAYOUT == TA);
  int slot0, num_tasks, stride = gridDim.x;
  // (four registers each for the counts and ends of up to 256 groups)
  [[maybe_unused]] GroupMap<4> map;
  if constexpr (ROWS) {
    map.count(p.g, TM, p.tiles_n);
    num_tasks = map.total;
  } else {
    num_tasks = p.num_tasks;
  }
  if constexpr (SHARES) {
    // (the first num_tasks % xcds shares hold one task more, as the first
    // gridDim.x % xcds XCDs hold one workgroup more: no share is without a
    // workgroup, and a grid of one workgroup per task does one each)
    const int xcds = min(p.num_xcds, (int)gridDim.x);
    const int xcd = blockIdx.x % xcds;
    const int share = num_tasks / xcds, more = num_tasks % xcds;
    const int first = xcd * share + min(xcd, more);
    slot0 = first + blockIdx.x / xcds;
    num_tasks = first + share + (xcd < more ? 1 : 0);
    stride = ((int)gridDim.x - xcd + xcds - 1) / xcds;
  } else if constexpr (ROWS) {
    // (the XCDs share the tiles there are, also where they are fewer than
    // the workgroups)
    const int busy = min((int)gridDim.x, num_tasks);
    if ((int)blockIdx.x >= busy) return;
    slot0 = xcd_slot(blockIdx.x, busy, p.num_xcds);
  } else {
    slot0 = xcd_slot(blockIdx.x, gridDim.x, p.num_xcds);
  }

  for (int task = slot0; task < num_tasks; task += stride) {
    int tm, tn;
    const bool part = SPLIT && task >= p.full_tasks;
    const int u = task - p.full_tasks;
    const int tile = part ? p.full_tasks + u % p.tiles : task;
    const int split = part ? u / p.tiles : 0;
    // the operands, rows and K of the task's product: the call's, or with
    // groups those of the tile's group
    const uint16_t *gA = p.A, *gB = p.B;
    uint16_t* gD = p.D;
    int row0 = 0, M = p.M, K = p.K, steps = p.split_steps;
    [[maybe_unused]] int group = 0;
    if constexpr (ROWS) {
      GroupTile t;
      map.find(p.g, task, TM, p.tiles_n, &t);
      group = t.group;
      row0 = t.beg;
      M = t.end;
      gB += group * p.g.stride;
      const int tiles_m = (M - row0 + TM - 1) / TM;
      tile_of_task(t.tile, tiles_m, p.tiles_n, min(tiles_m, p.group_m), &tm, &tn);
    } else if constexpr (GROUP) {
      const int per = p.tiles_m * p.tiles_n;
      group = tile / per;
      tile_of_task(tile - group * per, p.tiles_m, p.tiles_n, p.group_m, &tm, &tn);
      const int beg = group > 0 ? group_end(p.g, group - 1) : 0;
      K = max(group_end(p.g, group) - beg, 0);
      gA += (int64_t)beg * p.lda;
      gB += (int64_t)beg * p.ldb;
      gD += group * p.g.stride;
      if (SPLIT) steps = ((K + BK - 1) / BK + p.splits - 1) / p.splits;
    } else {
      tile_of_task(tile, p.tiles_m, p.tiles_n, p.group_m, &tm, &tn);
    }
    // this task's K steps
    const int nk = (K + BK - 1) / BK;
    const int kbeg = split * steps;
    const int kend = part ? min(nk, kbeg + steps) : nk;
    const int m0 = row0 + tm * TM;
    const int n0 = tn * TN;
    const int vm = min(TM, M - m0);    // valid rows of the A tile (A.T @ B: columns)
    const int vn = min(TN, p.N - n0);  // valid columns of D in this tile

    // MFMA operand layout (16 x 16 x 32): lane l holds row l % 16 of a
    // 16-row fragment and k = 8 (l / 16) .. +7 of the substep's 32
    const int lane = opaque_tid() & 63;
    const int l16 = lane & 15;
    const int lq = lane >> 4;

    // Accumulators start at zero.  The compiler places the zeroing just
    // before the K loop, after the prologue's barrier and fragment reads: at
    // least 30 instructions separate each register's reset from the first
    // (asm, so unguarded) MFMA that reads it, far more than the wait states
    // the hardware needs.  (Pinning it earlier, under the first loads, made
    // the register allocator spill.)
    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (f32x4){};
    fence();

    // Loader roles.  K-contiguous tiles: each wave instruction fills 1 KiB =
    // 8 rows of 128 B; wave w's instruction i of an operand with L loads per
    // thread covers rows (L w + i) * 8 ... +7, lane -> row lane/8 of the
    // group and a logical chunk by the swizzle (which depends on the row's
    // low four bits, i.e. on i's parity, L being even).
    // NN and TA B tile, TA A tile: each wave instruction fills 2 k rows of
    // 512 B, or 4 of 256 B where the tile is 128 wide.
    constexpr int A_RPL = 512 / TM, B_RPL = 512 / TN;  // k rows per wave instruction (512 or 256 B)
    const int nn_row_lo = lane / (64 / B_RPL);

    // Fragment read offsets (bytes within a stage).  Fragment f of a
    // K-contiguous tile (16 rows) sits 16 * 128 bytes after fragment 0: the
    // swizzle depends only on the row's low four bits.
    int fa[SUB], fb[SUB], fbn[NI];
    [[maybe_unused]] int fan[MI];
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      fa[s] = (wm * WTM + l16) * 128 + (((4 * s + lq) ^ swz_k(l16)) << 4);
      fb[s] = (wn * WTN + l16) * 128 + (((4 * s + lq) ^ swz_k(l16)) << 4);
    }
    {
      // transposing reads (NN B): in 16-lane block lq, lane i supplies row
      // k = 8 lq + i / 4 (+ 4 for the second read, + 32 per substep) and the
      // four columns n = wn*128 + 16 j + 4 (i % 4) .. +3, so that it receives
      // column 16 j + i at four consecutive k
      const int klane = 8 * lq + (l16 >> 2);
      // swz_n of every row this lane reads (the +4 and +32 row offsets of the
      // reads leave bits 0-1 and 3-4 of k unchanged)
      const int fl = swz_rows<TN>(klane);
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fbn[j] = klane * (2 * TN) + (((wn * (WTN / 8) + 2 * j + ((lane & 3) >> 1)) ^ fl) << 4) +
                 (lane & 1) * 8;
      if constexpr (LAYOUT == TA) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
          fan[i] = klane * (2 * TM) + (((wm * (WTM / 8) + 2 * i + ((lane & 3) >> 1)) ^ fl) << 4) +
                   (lane & 1) * 8;
      }
    }

    // Per-lane load offsets, fixed for the tile; the buffer descriptor of
    // each K step is rebased on that step (scalar work), so a load needs no
    // vector arithmetic.  Rows beyond M (A) or N (NT B) get an offset past
    // every range and read zeros.
    //
    // K steps: step s covers k = s*BK - koff .. +BK-1.  koff pads the first
    // step at its front so that the last one ends exactly at K8 (K rounded
    // up to 8; where K8 > K the operand is a zero-padded copy, or for the NN
    // B the descriptor ends at row K-1).  Only the first step reaches outside
    // [0, K8) -- below 0 -- so only its loads, issued in the prologue, need
    // per-lane masks.  (TA: k is a row of both operands, so no rounding.)
    const int K8 = LAYOUT == TA ? K : (K + 7) & ~7;
    const int koff = (BK - (K8 & (BK - 1))) & (BK - 1);
    // Groups of rows, A @ B.T: a tile starts its K steps at one of its own
    // and wraps around.  In step, all tiles would read the same 128 bytes of
    // rows a power of two apart, i.e. the same few memory channels: 64 groups
    // of 2 rows, N = 1024, K = 2048, weights from HBM, 67 -> 51 us (5.2
    // TB/s).  256-row tiles turn by group only, as the tiles of a row share
    // A's steps in L2 (16 groups of 1024, N = K = 4096: 507 us, 527 with a
    // turn per tile).
    [[maybe_unused]] int turn = 0;
    if constexpr (ROWS && LAYOUT == NT) {
      if (koff == 0 && nk > 0) turn = ((TM == BM ? 0 : tn * 5) + group * 3) % nk;
    }
    uint32_t a_off[DMA_PER_OPERAND], b_off[DMA_B];
    int kc[2];  // logical chunk of this lane for even / odd instruction index
#pragma unroll
    for (int h = 0; h < 2; ++h) kc[h] = (lane & 7) ^ swz_k(h * 8 + (lane >> 3));
#pragma unroll
    for (int i = 0; i < DMA_PER_OPERAND; ++i) {
      if constexpr (LAYOUT == TA) {
        const int k = A_RPL * (DMA_PER_OPERAND * wave + i) + nn_row_lo;
        a_off[i] = (uint32_t)(k * p.lda * 2 + ((lane & (64 / A_RPL - 1)) ^ swz_rows<TM>(k)) * 16);
      } else {
        const int r = (DMA_PER_OPERAND * wave + i) * 8 + (lane >> 3);
        a_off[i] = r < vm ? (uint32_t)(r * p.lda * 2 + kc[i & 1] * 16) : OOB;
      }
    }
    if (LAYOUT == NT) {
#pragma unroll
      for (int i = 0; i < DMA_B; ++i) {
        const int r = (DMA_B * wave + i) * 8 + (lane >> 3);
        b_off[i] = r < vn ? (uint32_t)(r * p.ldb * 2 + kc[i & 1] * 16) : OOB;
      }
    } else {
#pragma unroll
      for (int i = 0; i < DMA_B; ++i) {
        const int k = B_RPL * (DMA_B * wave + i) + nn_row_lo;
        const int c = (lane & (64 / B_RPL - 1)) ^ swz_rows<TN>(k);
        b_off[i] = (uint32_t)(k * p.ldb * 2 + c * 16);
      }
    }

    // LDS-DMA loads of K step ks into slot `slot` of its ring: the A tile (half 0)
    // or the B tile (half 1), issued one load at a time.  The descriptor
    // starts at the step's first column (K-contiguous tiles) or row (NN B)
    // and ends with the tile's last valid row, rounded up to a whole 8-element
    // chunk (where K or N is not a multiple of 8 the operand is a zero-padded
    // copy).  Steps at or past kend get an empty range: the slot is
    // zero-filled and the loop keeps a fixed pattern of loads in flight.
    struct Half {
      i32x4 r;
      uint32_t base;
      int k0;  // the step's first k (negative only for the first step)
    };
    // (Ranges are computed in 32 bits, which the argument check guarantees
    // suffice; 64-bit forms made the compiler branch inside the loop.)
    auto half_setup = [&](int ks, int slot, int half) {
      Half h;
      int kt = ks;
      if constexpr (ROWS && LAYOUT == NT) {
        kt += turn;
        kt -= kt >= nk ? nk : 0;
      }
      const int k0 = kt * BK - koff;
      const bool live = ks < kend;
      h.k0 = k0;
      h.base = lds0 + (half == EARLY ? 0 : RING2) + slot * (half == 0 ? A_BYTES : B_TILE) +
               ((half == 0 ? DMA_PER_OPERAND : DMA_B) * wave) * 1024;
      if ((half == 0 && LAYOUT != TA) || LAYOUT == NT) {
        // columns k0 .. K8 of the tile's rows
        const uint64_t src = half == 0 ? (uint64_t)(uintptr_t)(gA + (int64_t)m0 * p.lda)
                                       : (uint64_t)(uintptr_t)(gB + (int64_t)n0 * p.ldb);
        const int span = half == 0 ? (vm - 1) * p.lda : (vn - 1) * p.ldb;
        const uint32_t bytes = (uint32_t)(span + K8 - k0) * 2u;
        h.r = make_rsrc(src + 2 * (int64_t)k0, live ? bytes : 0u);
      } else if (half == 0) {
        // (TA) rows k0 .. min(k0 + BK, K) - 1 of A, columns m0 .. M (rounded up to 8)
        const int rows = min(BK, K - k0);
        const uint32_t bytes = (uint32_t)((rows - 1) * p.lda + ((M - m0 + 7) & ~7)) * 2u;
        h.r = make_rsrc((uint64_t)(uintptr_t)(gA + m0) + 2 * (int64_t)k0 * p.lda, live ? bytes : 0u);
      } else {
        // rows k0 .. min(k0 + BK, K) - 1 of B, columns n0 .. N (rounded up to 8)
        const int rows = min(BK, K - k0);
        const uint32_t bytes = (uint32_t)((rows - 1) * p.ldb + ((p.N - n0 + 7) & ~7)) * 2u;
        h.r = make_rsrc((uint64_t)(uintptr_t)(gB + n0) + 2 * (int64_t)k0 * p.ldb, live ? bytes : 0u);
      }
      return h;
    };
    // One load of a refill.  MASKED (prologue only): chunks or rows before
    // k = 0 read zeros.
    auto refill_one = [&](const Half& h, int half, int i, bool masked) {
      const uint32_t off = half == 0 ? a_off[i] : b_off[i];
      if ((half == 0 && LAYOUT != TA) || LAYOUT == NT) {
        dma16_at(h.r, !masked || h.k0 + (kc[i & 1] << 3) >= 0 ? off : OOB, h.base, i * 1024);
      } else {
        const int k = B_RPL * ((half == 0 ? DMA_PER_OPERAND : DMA_B) * wave + i) + nn_row_lo;
        dma16_at(h.r, !masked || h.k0 + k >= 0 ? off : OOB, h.base, i * 1024);
      }
      fence();
    };
    auto refill_stage = [&](int ks, int slot) {
      const Half ha = half_setup(ks, slot, 0);  // A and B slots agree for the first stages
      const Half hb = half_setup(ks, slot, 1);
#pragma unroll
      for (int i = 0; i < DMA_PER_OPERAND; ++i) refill_one(ha, 0, i, true);
#pragma unroll
      for (int i = 0; i < DMA_B; ++i) refill_one(hb, 1, i, true);
    };

    // Fragment reads of k-substep s of the stage in slot `slot`, one LDS
    // instruction at a time: the first A_READS items read the A fragments, the
    // rest the B fragments (one ds_read_b128 each from a K-contiguous tile,
    // two transposing reads from a tile of k rows).
    constexpr int A_READS = LAYOUT == TA ? 2 * MI : MI;
    constexpr int READS = A_READS + (LAYOUT == NT ? NI : 2 * NI);
    auto read_item = [&](int es, int ls, int s, Frags& F, int f) {
      const char* abase = smem + (EARLY == 0 ? es * A_BYTES : RING2 + ls * A_BYTES);
      const char* bbase = smem + (EARLY == 1 ? es * B_TILE : RING2 + ls * B_TILE);
      if (f < A_READS) {
        if constexpr (LAYOUT == TA) {
          const int i = f >> 1, h = f & 1;
          const u32x2 v = read_tr(abase + fan[i] + (s * 32 + 4 * h) * (2 * TM));
          F.a[i][2 * h] = v[0];
          F.a[i][2 * h + 1] = v[1];
        } else {
          F.a[f] = *(const u32x4*)(abase + fa[s] + f * 2048);
        }
      } else if (LAYOUT == NT) {
        const int j = f - A_READS;
        F.b[j] = *(const u32x4*)(bbase + fb[s] + j * 2048);
      } else {
        const int j = (f - A_READS) >> 1, h = (f - A_READS) & 1;
        const u32x2 v = read_tr(bbase + fbn[j] + (s * 32 + 4 * h) * (2 * TN));
        F.b[j][2 * h] = v[0];
        F.b[j][2 * h + 1] = v[1];
      }
    };
    // All reads of a substep in item order.  The fences keep that order: the
    // loop head then sees the same sequence of outstanding reads from the
    // prologue as from the loop's back edge, and waits only for the ones the
    // first MFMAs need.
    auto read_frags = [&](int es, int ls, int s, Frags& F) {
#pragma unroll
      for (int f = 0; f < READS; ++f) {
        read_item(es, ls, s, F, f);
        fence();
      }
    };
    // the share of `total` items due before step q of `steps`, spread evenly
    auto share = [](int q, int steps, int total, auto&& item) {
#pragma unroll
      for (int f = (q * total) / steps; f < ((q + 1) * total) / steps; ++f) item(f);
    };

    // Operand order (B fragment first) leaves each lane holding one row of D
    // and four consecutive columns.  Consecutive MFMAs share a B fragment, so
    // the next substep's reads (A fragments first, then B) arrive in the
    // order its MFMAs need them; the A fragments run forwards under even B
    // fragments and backwards under odd ones, so each MFMA changes one
    // operand only.
    auto mfma_pair = [&](const Frags& F, int q) {
#pragma unroll
      for (int t = 2 * q; t < 2 * q + 2; ++t) {
        const int j = t / MI, i = (j & 1) ? MI - 1 - t % MI : t % MI;
        mfma16<T>(acc[i][j], F.b[j], F.a[i]);
      }
    };

    // The rings (AHEAD = 2; with more, the rings have AHEAD + 1 and AHEAD
    // slots, and "ks+2" below reads "ks+AHEAD", the stages between in
    // flight): stage ks (counted from the task's first step) keeps its
    // EARLY operand's tile in slot ks % 3 of the three-slot ring and the
    // other's in slot ks % 2 of the two-slot ring.  Entering step ks, stage
    // ks has landed, stage ks+1 is in flight, and F0 holds substep 0 of
    // stage ks.  Substep 0 runs its 64 MFMAs in pairs with the reads of
    // substep 1 spread between them (spread, not bunched: a burst of reads
    // fills the LDS command queue and stalls the MFMA issue behind it), and
    // with the loads of stage ks+2's EARLY tile: its slot held stage ks-1,
    // which every wave finished reading before the last barrier.  Substep 1
    // runs BAR_PAIR pairs, then the barrier: stage ks+1 has landed for every
    // wave (only the 8 EARLY loads just issued may be in flight: loads
    // complete in order) and every wave is done reading stage ks, so the rest
    // of substep 1 interleaves the reads of stage ks+1's first substep with
    // the loads of stage ks+2's other tile into stage ks's two-ring slot.
    // The third slot spreads a stage's loads over the whole step instead of
    // its second half, halving the requests in flight at a time (measured:
    // 3-4% faster on the large and ragged shapes).
    Frags F0, F1;
    refill_stage(kbeg, 0);
    refill_stage(kbeg + 1, 1);
    if constexpr (AHEAD > 2) {
      refill_stage(kbeg + 2, 2);
      refill_stage(kbeg + 3, 3);
    }
    wait_vm_barrier<(AHEAD - 1) * (DMA_PER_OPERAND + DMA_B)>();
    read_frags(0, 0, 0, F0);

    // Column sums of A: a lane adds the eight k that it holds of each A
    // fragment.  All tiles of a tile row read the same A, so they share the
    // K steps: step ks is added by wave column ks mod (2 tiles_n) of the
    // row's 2 tiles_n (two to a tile), between the substeps, where both
    // substeps' fragments are at hand.  (One v_dot2c per fragment word in
    // every tile and step took 8 to 12% of 5120 x 8192 x 8192; a branch per
    // step costs nothing measurable.)
    [[maybe_unused]] float cs[MI];
    [[maybe_unused]] int sum_at = 0;
    if constexpr (SUMS) {
#pragma unroll
      for (int i = 0; i < MI; ++i) cs[i] = 0.0f;
      const int period = 2 * p.tiles_n;
      sum_at = kbeg + (2 * tn + wn + period - kbeg % period) % period;
    }
    int es = 0;  // early-ring slot of stage ks
    for (int ks = kbeg; ks < kend; ++ks) {
      const int ls = (ks - kbeg) & (AHEAD - 1);     // other-ring slot of stage ks
      const int es1 = es == AHEAD ? 0 : es + 1;     // early-ring slot of stage ks+1
      // early-ring slot of stage ks+AHEAD (that of stage ks-1)
      const int es2 = AHEAD == 2 ? (es1 == 2 ? 0 : es1 + 1) : (es == 0 ? AHEAD : es - 1);
      Half he;
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        share(q, PAIRS, READS, [&](int f) { read_item(es, ls, 1, F1, f); });
        mfma_pair(F0, q);
        fence();
        // (the descriptor's scalar work goes behind the first MFMAs)
        if (q == 0) he = half_setup(ks + AHEAD, es2, EARLY);
        // stages from the third on start at k >= 0: no masks
        share(q, PAIRS, DMA_E, [&](int i) { refill_one(he, EARLY, i, false); });
      }
      if constexpr (SUMS) {
        if (ks == sum_at) {
          sum_at += 2 * p.tiles_n;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < MI; ++i) cs[i] = sum2<T>(cs[i], F0.a[i][k]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < MI; ++i) cs[i] = sum2<T>(cs[i], F1.a[i][k]);
        }
        fence();
      }
      const Half hl = half_setup(ks + AHEAD, ls, 1 - EARLY);
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        if (q == BAR_PAIR) {
          wait_vm_barrier<(AHEAD - 2) * (DMA_E + DMA_L) + DMA_E>();
          fence();
        }
        if (q >= BAR_PAIR)
          share(q - BAR_PAIR, PAIRS - BAR_PAIR, READS,
                [&](int f) { read_item(es1, AHEAD == 2 ? ls ^ 1 : (ls + 1) & (AHEAD - 1), 0, F0, f); });
        mfma_pair(F1, q);
        fence();
        if (q >= BAR_PAIR)
          share(q - BAR_PAIR, PAIRS - BAR_PAIR, DMA_L,
                [&](int i) { refill_one(hl, 1 - EARLY, i, false); });
      }
      es = es1;
    }

    wait_vm_barrier<0>();  // every wave is done with the ring; reuse it for staging
    // wait states between the last MFMAs and the first reads of their results
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    fence();

    if constexpr (SUMS) {
      // the four lane groups' sums of each column, added in a fixed order;
      // column_sums adds those of the tile row's wave columns
      float* w = p.colsum_ws + ((size_t)task * 2 + wn) * TM + wm * WTM;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        float s = cs[i];
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lq == 0) w[16 * i + l16] = s;
      }
    }

    if (!EPI && part) {
      // FP32 partial tile, row-major 256 x 256: lane holds row l16 of each
      // 16-row block and columns j*16 + 4*lq .. +3 (16 contiguous bytes);
      // 16 x 16 blocks wholly outside D are skipped (nothing reads them)
      float* w = p.ws + (size_t)(split * p.tiles + u % p.tiles) * (TM * TN) +
                 (size_t)(wm * WTM + l16) * TN + wn * WTN + 4 * lq;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (wm * WTM + i * 16 >= vm) break;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (wn * WTN + j * 16 >= vn) break;
          *(float4*)(w + i * 16 * TN + j * 16) =
              make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      continue;
    }

    if constexpr (EPI) {
      // Epilogue of a layer's product (epilogue.h): per 32-row band (two
      // 16-row blocks), the band's FP32 accumulators of this wave are staged
      // in LDS (rows of CHF 16-byte chunks), so that each lane gets eight
      // consecutive columns of a row and reads the residual or Z, and writes
      // Z and D, in 16-byte accesses.  (Staged in 16 bits, as below, the
      // residual could only be added after a first rounding.)  Chunk c of
      // row r is stored at c ^ (c >> 3 & 1) ^ (r & 7): the writes (one chunk
      // of eight rows) and the reads (every other chunk of a row) both touch
      // distinct banks.  The loop over the passes is not unrolled: the code of
      // eight activations and slopes stays small enough for the instruction
      // cache beside the K loop.  A pass reads the next one's residual or Z
      // from memory before it computes, and where a wave has its SIMD to
      // itself (nothing else would cover the latency) the next one's values
      // from LDS too: 4096^3 without an activation 103 -> 97 us; with two
      // workgroups per CU the registers that takes cost more (48 ragged
      // groups, 53 us against 56).
      constexpr int CH = WTN / 8;      // lanes per staged row
      constexpr int CHF = WTN / 4;     // 16-byte chunks per staged row
      constexpr int RPI = 64 / CH;     // rows per wave instruction
      constexpr int R = 4;             // row instructions per pass
      constexpr int PASSES = 32 / (RPI * R);  // passes per band
      static_assert(WAVES * 32 * WTN * 4 <= LDS_BYTES, "a band of every wave fits the rings");
      const Epilogue& ep = p.e;
      char* stg = smem + wave * (32 * CHF * 16);
      const int cc = lane % CH, rl = lane / CH;
      const int col = n0 + wn * WTN + cc * 8;
      const int rowb = m0 + wm * WTM + rl;  // this lane's first row of the wave's
      uint32_t bias[4] = {0u, 0u, 0u, 0u};
      if (!ep.grad && ep.bias != nullptr && col < p.N)
        load_row<4>(ep.bias + group * ep.bias_stride, col, p.N, bias);
      // the operand each output needs: the residual, or the gradient's Z
      const uint16_t* side = ep.grad ? ep.z : ep.res;
      const int64_t lds_ = ep.grad ? ep.ldz : ep.ldr;
      auto fetch = [&](int pass, uint32_t(&w)[R][4]) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int row = rowb + (pass * R + t) * RPI;
#pragma unroll
          for (int k = 0; k < 4; ++k) w[t][k] = 0u;
          if (side != nullptr && !part && row < M && col < p.N)
            load_row<4>(side + row * lds_, col, p.N, w[t]);
        }
      };
      auto stage = [&](int band) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = half * 16 + l16;
#pragma unroll
          for (int j = 0; j < NI; ++j) {
            const int c = 4 * j + lq;
            *(f32x4*)(stg + ((r * CHF + (c ^ ((c >> 3) & 1) ^ (r & 7))) << 4)) =
                acc[2 * band + half][j];
          }
        }
      };
      uint32_t w[R][4], w_next[R][4] = {};
      fetch(0, w);
      stage(0);
      // Loads are waited for on every path (the empty asm uses their
      // results): one that the compiler believes pending when the next tile's
      // K loop begins makes it wait for all loads inside that loop.
      asm volatile("" : "+v"(bias[0]), "+v"(bias[1]), "+v"(bias[2]), "+v"(bias[3]));
#pragma unroll
      for (int t = 0; t < R; ++t)
        asm volatile("" : "+v"(w[t][0]), "+v"(w[t][1]), "+v"(w[t][2]), "+v"(w[t][3]));
      auto read_staged = [&](int pass, float(&v)[R][8]) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int r = (pass % PASSES * R + t) * RPI + rl;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 2 * cc + h;
            const f32x4 x = *(const f32x4*)(stg + ((r * CHF + (c ^ ((c >> 3) & 1) ^ (r & 7))) << 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[t][4 * h + k] = x[k];
          }
        }
      };
      constexpr bool PIPE = per_cu<LAYOUT, SPLIT, TN, TM, EPI, GROUP>() == 1;
      float v[R][8];
      [[maybe_unused]] float v_next[R][8];
      if constexpr (PIPE) read_staged(0, v);
#pragma unroll 1
      for (int pass = 0; pass < (MI / 2) * PASSES; ++pass) {
        // (a wave's LDS accesses complete in order: the next band's writes
        // follow the reads of this one's last values)
        const int to_stage = PIPE ? pass + 1 : pass;  // the pass whose band to stage now
        if (to_stage % PASSES == 0) {
          switch (to_stage / PASSES) {
            case 1: stage(1); break;
            case 2: if constexpr (MI > 4) stage(2); break;
            case 3: if constexpr (MI > 4) stage(3); break;
            default: break;
          }
        }
        if (pass + 1 < (MI / 2) * PASSES) {
          fetch(pass + 1, w_next);
          if constexpr (PIPE) read_staged(pass + 1, v_next);
        }
        if constexpr (!PIPE) read_staged(pass, v);
        if (part) {
          // the part's FP32 partial tile, row-major TM x TN (elements outside
          // D are skipped: nothing reads them)
          float* part_ws = p.ws + (size_t)(split * p.tiles + u % p.tiles) * (TM * TN) +
                           wn * WTN + cc * 8;
#pragma unroll
          for (int t = 0; t < R; ++t) {
            const int r = wm * WTM + rl + (pass * R + t) * RPI;
            if (m0 + r < M && col < p.N) {
              *(f32x4*)(part_ws + r * TN) = (f32x4){v[t][0], v[t][1], v[t][2], v[t][3]};
              *(f32x4*)(part_ws + r * TN + 4) = (f32x4){v[t][4], v[t][5], v[t][6], v[t][7]};
            }
          }
        } else if (ep.grad) {
          apply_slope<T>(ep.act, v, w);
        } else {
#pragma unroll
          for (int t = 0; t < R; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[t][k] += unpack<T>(bias[k >> 1], k & 1);
          if (ep.z != nullptr) {
#pragma unroll
            for (int t = 0; t < R; ++t) {
              const int row = rowb + (pass * R + t) * RPI;
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = pack2<T>(v[t][2 * k], v[t][2 * k + 1]);
              if (row < M && col < p.N)
                store_row<4>(ep.z + (int64_t)row * ep.ldz, col, p.N, o);
            }
          }
          apply_act(ep.act, v);
          if (ep.res != nullptr) {
#pragma unroll
            for (int t = 0; t < R; ++t)
#pragma unroll
              for (int k = 0; k < 8; ++k) v[t][k] += unpack<T>(w[t][k >> 1], k & 1);
          }
        }
#pragma unroll
        for (int t = 0; t < R; ++t)
          asm volatile("" : "+v"(w_next[t][0]), "+v"(w_next[t][1]), "+v"(w_next[t][2]),
                       "+v"(w_next[t][3]));
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int row = rowb + (pass * R + t) * RPI;
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = pack2<T>(v[t][2 * k], v[t][2 * k + 1]);
          if (!part && row < M && col < p.N)
            store_row<4>(gD + (int64_t)row * p.ldd, col, p.N, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[t][k] = w_next[t][k];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if constexpr (PIPE) v[t][k] = v_next[t][k];
        }
      }
      wait_lds_barrier();
      continue;
    }

    // Epilogue: per 32-row band (two 16-row blocks), round, stage the band's
    // 32 x WTN outputs of this wave in LDS (rows of CH 16-byte chunks,
    // swizzled by row), then store 16-byte row chunks.  Each phase is issued
    // whole before the next (all conversions into registers of their own,
    // all LDS writes, all read-backs, then the stores), so that their
    // latencies overlap instead of adding up per chunk.
    constexpr int CH = WTN / 8;       // 16-byte chunks per staged row
    constexpr int RPI = 64 / CH;      // rows per wave instruction of the read-back
    constexpr int NR = 32 / RPI;      // read-back instructions per band
    char* stg = smem + wave * (32 * CH * 16);
    // (the layer products' 16-byte stores take D rows of any alignment)
    const bool interior = p.d_vec && vm == TM && vn == TN;
#pragma unroll
    for (int band = 0; band < MI / 2; ++band) {
      // lane holds row half*16 + l16 of the band, columns j*16 + 4*lq + 0..3
      // of each block j: 16-byte chunk 2j + lq/2, its lower or upper 8 bytes
      u32x2 v[2][NI];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          v[half][j][0] = pack2<T>(acc[2 * band + half][j][0], acc[2 * band + half][j][1]);
          v[half][j][1] = pack2<T>(acc[2 * band + half][j][2], acc[2 * band + half][j][3]);
        }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = half * 16 + l16;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int chunk = 2 * j + (lq >> 1);
          *(u32x2*)(stg + row * (CH * 16) + ((chunk ^ (row & (CH - 1))) << 4) + (lq & 1) * 8) =
              v[half][j];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      const int rowb = m0 + wm * WTM + band * 32;
      const int col0 = n0 + wn * WTN;
      const int cc = lane % CH;
      u32x4 r[NR];
#pragma unroll
      for (int t = 0; t < NR; ++t) {
        const int rr = t * RPI + lane / CH;
        r[t] = *(const u32x4*)(stg + rr * (CH * 16) + ((cc ^ (rr & (CH - 1))) << 4));
      }
      __builtin_amdgcn_sched_barrier(0);
      // D is written once and not read again here: non-temporal stores
      // (measured 0.3-1% faster, 4.7% on the large FP8 product)
      if (interior) {
        // the whole tile is inside D and its rows are 16-byte aligned
#pragma unroll
        for (int t = 0; t < NR; ++t) {
          const int rr = t * RPI + lane / CH;
          __builtin_nontemporal_store(r[t],
                                      (u32x4_any*)(gD + (int64_t)(rowb + rr) * p.ldd + col0 + cc * 8));
        }
      } else {
#pragma unroll
        for (int t = 0; t < NR; ++t) {
          const int rr = t * RPI + lane / CH;
          const int row = rowb + rr;
          const int col = col0 + cc * 8;
          if (row < M && col < p.N) {
            uint16_t* dst = gD + (int64_t)row * p.ldd + col;
            if (p.d_vec && col + 8 <= p.N) {
              __builtin_nontemporal_store(r[t], (u32x4_any*)dst);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (col + e < p.N) dst[e] = (uint16_t)(r[t][e >> 1] >> ((e & 1) * 16));
            }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // staging reads done before the next tile refills the ring; the stores
    // drain while the next tile's first loads are in flight
    wait_lds_barrier();
  }
}

}  // namespace dg
