// layer_kernel.h -- the tiled kernel of a layer's products on the MI355X
// (gfx950): D = A @ B.T, A @ B (with an epilogue) and A.T @ B (with A's column
// sums), for one matrix or one per group of rows.
//
// The product is computed as in gemm_kernel.h, whose comments explain what
// the two have in common: 256 x 256 tiles of four 128 x 128 waves on
// v_mfma_f32_16x16x32, 64-deep K stages loaded by LDS-DMA into two rings, XOR
// swizzles, ragged edges masked by buffer ranges, split-K through FP32 partial
// tiles.  What differs:
//   * layout TA: A and B both have k as their row, so both tiles are 64 k
//     rows, read with transposing LDS reads;
//   * 128 x 128 tiles, two workgroups to a CU, or one with deeper rings;
//   * A.T @ B finds its next tile and starts that tile's first loads before
//     it writes the last one's outputs, so that the loads' latency lies under
//     the epilogue (the stores have until the barrier in the next tile's first
//     step, whose counted wait includes them);
//   * the epilogue works on FP32 values staged in LDS (epilogue.h);
//   * row groups (groups.h): the tiles' places and K come from the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cdna_ops.h"
#include "epilogue.h"
#include "groups.h"
#include "i8.h"
#include "tile_config.h"
#include "tile_sched.h"

namespace dg {

struct LayerParams {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* D;
  int M, N, K;
  int lda, ldb, ldd;
  int tiles_m, tiles_n, group_m, num_tasks, num_xcds;
  // split-K (the SPLIT kernels), as in gemm_kernel.h: tasks below full_tasks
  // are whole tiles, task full_tasks + u is part u / tiles of tile full_tasks
  // + u % tiles, whose FP32 partial tile lies at ws + (part * tiles + u %
  // tiles) * TM * TN.  With groups (TA) the parts divide each group's K.
  int full_tasks, splits, split_steps, tiles;
  float* ws;
  Epilogue e;
  Groups g;
  // SUMS: each task leaves its two wave columns' FP32 sums of its TM columns
  // of A at colsum_ws + task * 2 TM (added up by column_sums.h); or, where
  // colsum_ws is null, the first tile of each tile row writes its columns of
  // colsum (M a group)
  float* colsum_ws;
  uint16_t* colsum;
};

// The int8 products (i8.h): A, B, K, lda, ldb and the groups' stride count pairs
// of int8 values.
struct LayerI8Params : LayerParams {
  I8Scales s;
};

// Stages loaded ahead of the one in use.  Two, with rings of three slots for
// one operand and two for the other, fill the LDS for 256-wide tiles.  128 x
// 128 tiles are 80 KiB that way:
//   * many tiles run two workgroups per CU, so that one computes while the
//     other waits for its first tiles or writes its last ones;
//   * at most one tile or part per CU (the SPLIT kernels) runs four stages
//     ahead instead, in 144 KiB, to cover the load latency alone (a K step
//     of 512 x 512 x 4096, A @ B.T: 0.47 -> 0.34 us).
template <bool SPLIT, int TN, int TM>
constexpr int stages_ahead() { return SPLIT && TM == BM / 2 && TN == BN / 2 ? 4 : 2; }
template <bool SPLIT, int TN, int TM>
constexpr int per_cu() { return !SPLIT && TM == BM / 2 && TN == BN / 2 ? 2 : 1; }

// A task's tile: operands, rows and K of its product (the call's, or its
// group's), place and K steps.  All values are the same in every lane.
struct TileAt {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* D;
  int M, K;          // end of the rows (TA: columns of A), K
  int m0, n0;        // first row and column
  int vm, vn;        // rows and columns inside
  int tn, group;
  int nk, kbeg, kend;  // K steps of the product, and the task's
  int koff, K2;        // K in whole words; the first step starts at k = -koff
  int turn;            // step s reads step (s + turn) mod nk
  int task, part, part_index;  // part: a part of a split tile, at part_index in ws
};

// T: element type; LAYOUT NT, NN or TA; SPLIT: tasks may be parts of K; TN,
// TM: tile columns and rows; GROUP: row groups (NT, NN: groups of rows of A
// and D with a B each; TA: sums over a group's rows, a D per group); SUMS:
// (TA) column sums of A.  NT and NN apply the epilogue p.e.
// T I8<O>: int8 operands (NT alone) and results of type O, the accumulators
// whole numbers in the same registers.
template <typename T, int LAYOUT, bool SPLIT, int TN, int TM, bool GROUP, bool SUMS = false>
__global__ __launch_bounds__(THREADS, (per_cu<SPLIT, TN, TM>())) void layer_gemm_kernel(
    std::conditional_t<is_i8<T>, LayerI8Params, LayerParams> p) {
  using O = output_of<T>;
  static_assert(!is_i8<T> || LAYOUT == NT, "int8 operands are rows of K values");
  static_assert(BK == 64, "the swizzles and offsets below assume 128-byte rows of k");
  static_assert(LAYOUT != TA || TM == TN, "A.T @ B takes square tiles");
  static_assert(!SUMS || LAYOUT == TA, "column sums of A where its rows are k");
  static_assert(!(GROUP && SPLIT && LAYOUT != TA), "row groups of A are not split in K");
  constexpr bool EPI = LAYOUT != TA;
  constexpr bool ROWS = GROUP && LAYOUT != TA;
  constexpr int SUB = BK / 32;             // 32-deep MFMA substeps per stage
  constexpr int BAR_PAIR = 2;              // MFMA pairs of the last substep before its barrier
  constexpr int WTM = TM / 2, WTN = TN / 2;  // wave tile
  constexpr int MI = WTM / 16, NI = WTN / 16;
  constexpr int PAIRS = MI * NI / 2;       // MFMA pairs per substep
  constexpr int A_BYTES = TM * BK * 2, B_BYTES = TN * BK * 2;
  constexpr int DMA_A = A_BYTES / (THREADS * 16), DMA_B = B_BYTES / (THREADS * 16);
  // the operand whose loads are issued first, with one ring slot more
  constexpr int EARLY = LAYOUT == NT ? 0 : 1;
  constexpr int DMA_E = EARLY == 0 ? DMA_A : DMA_B, DMA_L = EARLY == 0 ? DMA_B : DMA_A;
  constexpr int E_BYTES = EARLY == 0 ? A_BYTES : B_BYTES, L_BYTES = EARLY == 0 ? B_BYTES : A_BYTES;
  constexpr int AHEAD = stages_ahead<SPLIT, TN, TM>();
  constexpr int RING2 = (AHEAD + 1) * E_BYTES, RINGS = RING2 + AHEAD * L_BYTES;
  // Staging of the outputs: 16 rows of every wave in FP32 (EPI) or 32 in 16
  // bits, in the early ring's last slot, which the next tile's first stages
  // leave free (where that slot is too small, behind the rings).
  constexpr int STAGING = WAVES * 16 * WTN * 4;
  constexpr int STAGE_AT = STAGING <= E_BYTES ? AHEAD * E_BYTES : RINGS;
  constexpr int LDS_BYTES = STAGING <= E_BYTES ? RINGS : RINGS + STAGING;
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
  const uint32_t lds0 = lds_addr(smem);

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;  // wave tile row and column

  // Where all tasks are alike, each XCD gets one run of them, an even share,
  // which its workgroups take in turn: the tasks of a last, partial round
  // then fall on all XCDs, a few CUs each (48 groups, 5003 rows, 63 -> 53 us;
  // A.T @ B 5120 x 8192 x 8192, 2.5 rounds, 551 -> 533).  Else the tasks are
  // dealt round by round, so that a round's tiles are neighbours over all
  // XCDs: groups of different K would leave the XCDs with different work (16
  // groups' A.T @ B 508 us, 1254 in runs), and 16 groups of 1024 rows take
  // 509 us, 523 in runs.
  constexpr bool SHARES = !SPLIT && (GROUP ? ROWS && TM == BM / 2 : true);
  int task, num_tasks, stride = gridDim.x;
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
    task = first + blockIdx.x / xcds;
    num_tasks = first + share + (xcd < more ? 1 : 0);
    stride = ((int)gridDim.x - xcd + xcds - 1) / xcds;
  } else {
    // (with groups of rows the XCDs share the tiles there are, also where
    // they are fewer than the workgroups)
    const int busy = ROWS ? min((int)gridDim.x, num_tasks) : (int)gridDim.x;
    if ((int)blockIdx.x >= busy) return;
    task = xcd_slot(blockIdx.x, busy, p.num_xcds);
  }
  if (task >= num_tasks) return;

  auto locate = [&](int task) {
    TileAt t;
    t.task = task;
    t.part = SPLIT && task >= p.full_tasks;
    const int u = task - p.full_tasks;
    const int tile = t.part ? p.full_tasks + u % p.tiles : task;
    const int split = t.part ? u / p.tiles : 0;
    t.part_index = t.part ? split * p.tiles + u % p.tiles : 0;
    t.A = p.A;
    t.B = p.B;
    t.D = p.D;
    t.M = p.M;
    t.K = p.K;
    t.group = 0;
    int tm, row0 = 0, steps = p.split_steps;
    if constexpr (ROWS) {
      GroupTile g;
      map.find(p.g, task, TM, p.tiles_n, &g);
      t.group = g.group;
      row0 = g.beg;
      t.M = g.end;
      t.B += g.group * p.g.stride;
      const int tiles_m = (g.end - g.beg + TM - 1) / TM;
      tile_of_task(g.tile, tiles_m, p.tiles_n, min(tiles_m, p.group_m), &tm, &t.tn);
    } else if constexpr (GROUP) {
      const int per = p.tiles_m * p.tiles_n;
      t.group = tile / per;
      tile_of_task(tile - t.group * per, p.tiles_m, p.tiles_n, p.group_m, &tm, &t.tn);
      const int beg = t.group > 0 ? group_end(p.g, t.group - 1) : 0;
      t.K = max(group_end(p.g, t.group) - beg, 0);
      t.A += (int64_t)beg * p.lda;
      t.B += (int64_t)beg * p.ldb;
      t.D += t.group * p.g.stride;
      if (SPLIT) steps = ((t.K + BK - 1) / BK + p.splits - 1) / p.splits;
    } else {
      tile_of_task(tile, p.tiles_m, p.tiles_n, p.group_m, &tm, &t.tn);
    }
    t.nk = (t.K + BK - 1) / BK;
    t.kbeg = split * steps;
    t.kend = t.part ? min(t.nk, t.kbeg + steps) : t.nk;
    t.m0 = row0 + tm * TM;
    t.n0 = t.tn * TN;
    t.vm = min(TM, t.M - t.m0);
    t.vn = min(TN, p.N - t.n0);
    // (an odd row of K values is a copy padded with a zero; TA: k is a row of
    // both operands, so K is not rounded up)
    t.K2 = LAYOUT == TA ? t.K : (t.K + 1) & ~1;
    t.koff = (BK - (t.K2 & (BK - 1))) & (BK - 1);
    // Groups of rows, A @ B.T: a tile starts its K steps at one of its own
    // and wraps around.  In step, all tiles would read the same 128 bytes of
    // rows a power of two apart, i.e. the same few memory channels: 64 groups
    // of 2 rows, N = 1024, K = 2048, weights from HBM, 67 -> 51 us (5.2
    // TB/s).  256-row tiles turn by group only, as the tiles of a row share
    // A's steps in L2 (16 groups of 1024, N = K = 4096: 507 us, 527 with a
    // turn per tile).
    t.turn = 0;
    // (K a multiple of 64 alone: the step that begins below k = 0 has to be the
    // first, the only one whose loads are masked.)
    if constexpr (ROWS && LAYOUT == NT) {
      if (t.koff == 0 && t.nk > 0) t.turn = ((TM == BM ? 0 : t.tn * 5) + t.group * 3) % t.nk;
    }
    return t;
  };

  // Loader roles.  K-contiguous tiles: a wave instruction fills 8 rows of 128
  // B, wave w's instruction i of an operand with L loads per thread rows (L w
  // + i) * 8 ... +7.  Tiles of k rows: 2 rows of 512 B, or 4 of 256 B where
  // the tile is 128 wide.  The offsets are fixed for a tile; the descriptor
  // is rebased on each K step.
  constexpr int A_RPL = 512 / TM, B_RPL = 512 / TN;
  TileAt at = locate(task);
  uint32_t a_off[DMA_A], b_off[DMA_B];
  auto set_offsets = [&](int lane) {
#pragma unroll
    for (int i = 0; i < DMA_A; ++i) {
      if constexpr (LAYOUT == TA) {
        const int k = A_RPL * (DMA_A * wave + i) + lane / (64 / A_RPL);
        a_off[i] = (uint32_t)(k * p.lda * 2 + ((lane & (64 / A_RPL - 1)) ^ swz_rows<TM>(k)) * 16);
      } else {
        const int r = (DMA_A * wave + i) * 8 + (lane >> 3);
        const int kc = (lane & 7) ^ swz_k((i & 1) * 8 + (lane >> 3));
        a_off[i] = r < at.vm ? (uint32_t)(r * p.lda * 2 + kc * 16) : OOB;
      }
    }
#pragma unroll
    for (int i = 0; i < DMA_B; ++i) {
      if constexpr (LAYOUT == NT) {
        const int r = (DMA_B * wave + i) * 8 + (lane >> 3);
        const int kc = (lane & 7) ^ swz_k((i & 1) * 8 + (lane >> 3));
        b_off[i] = r < at.vn ? (uint32_t)(r * p.ldb * 2 + kc * 16) : OOB;
      } else {
        const int k = B_RPL * (DMA_B * wave + i) + lane / (64 / B_RPL);
        b_off[i] = (uint32_t)(k * p.ldb * 2 + ((lane & (64 / B_RPL - 1)) ^ swz_rows<TN>(k)) * 16);
      }
    }
  };

  // LDS-DMA loads of K step ks of A (half 0) or B (half 1) into a ring slot;
  // steps at or past kend load zeros (an empty range).
  struct Half {
    i32x4 r;
    uint32_t base;
    int k0;
  };
  auto half_setup = [&](int ks, int slot, int half) {
    Half h;
    int kt = ks;
    if constexpr (ROWS && LAYOUT == NT) {
      kt += at.turn;
      kt -= kt >= at.nk ? at.nk : 0;
    }
    const int k0 = kt * BK - at.koff;
    const bool live = ks < at.kend;
    h.k0 = k0;
    h.base = lds0 + (half == EARLY ? 0 : RING2) + slot * (half == 0 ? A_BYTES : B_BYTES) +
             ((half == 0 ? DMA_A : DMA_B) * wave) * 1024;
    if (half == 0 ? LAYOUT != TA : LAYOUT == NT) {
      // columns k0 .. K2 of the tile's rows
      const uint64_t src = half == 0 ? (uint64_t)(uintptr_t)(at.A + (int64_t)at.m0 * p.lda)
                                     : (uint64_t)(uintptr_t)(at.B + (int64_t)at.n0 * p.ldb);
      const int span = half == 0 ? (at.vm - 1) * p.lda : (at.vn - 1) * p.ldb;
      const uint32_t bytes = (uint32_t)(span + at.K2 - k0) * 2u;
      h.r = make_rsrc(src + 2 * (int64_t)k0, live ? bytes : 0u);
    } else {
      // rows k0 .. min(k0 + BK, K) - 1, columns m0 .. M or n0 .. N (rounded up
      // to whole words: the range check is by word; an odd row is a padded copy)
      const int ld = half == 0 ? p.lda : p.ldb;
      const int cols = half == 0 ? at.M - at.m0 : p.N - at.n0;
      const int rows = min(BK, at.K - k0);
      const uint32_t bytes = (uint32_t)((rows - 1) * ld + ((cols + 1) & ~1)) * 2u;
      const uint64_t src = half == 0 ? (uint64_t)(uintptr_t)(at.A + at.m0)
                                     : (uint64_t)(uintptr_t)(at.B + at.n0);
      h.r = make_rsrc(src + 2 * (int64_t)k0 * ld, live ? bytes : 0u);
    }
    return h;
  };
  // One load.  (Only the first step reaches below k = 0; its loads are masked
  // here, by lane, in the prologue.)
  auto refill_one = [&](const Half& h, int half, int i, int lane, bool masked) {
    const uint32_t off = half == 0 ? a_off[i] : b_off[i];
    int k;  // the lane's first k within the step
    if (half == 0 ? LAYOUT != TA : LAYOUT == NT)
      k = ((lane & 7) ^ swz_k((i & 1) * 8 + (lane >> 3))) << 3;
    else
      k = half == 0 ? A_RPL * (DMA_A * wave + i) + lane / (64 / A_RPL)
                    : B_RPL * (DMA_B * wave + i) + lane / (64 / B_RPL);
    dma16_at(h.r, !masked || h.k0 + k >= 0 ? off : OOB, h.base, i * 1024);
    fence();
  };
  // The first K step of a K-contiguous operand where its 16-byte pieces
  // straddle k = 0: word by word, those before it zero.  (So rows of K values
  // need no padded copy for their last piece: A @ B.T 4096 x 4096 x 4098
  // 133 -> 112 us.)
  auto first_words = [&](const Half& h, int half, int lane) {
    const int loads = half == 0 ? DMA_A : DMA_B, ld = half == 0 ? p.lda : p.ldb;
    const int rows = half == 0 ? at.vm : at.vn;
#pragma unroll 1
    for (int j = 0; j < 4 * loads; ++j) {
      // the word that this lane fills of the 64 lanes' pieces of load j / 4
      const int i = j >> 2, l = (j & 3) * 16 + (lane >> 2);
      const int r = (loads * wave + i) * 8 + (l >> 3);
      const int k = (((l & 7) ^ swz_k((i & 1) * 8 + (l >> 3))) << 3) + 2 * (lane & 3);
      dma4_at(h.r, r < rows && h.k0 + k >= 0 ? (uint32_t)(r * ld + k) * 2u : OOB, h.base + j * 256, 0);
      fence();
    }
  };
  auto prologue = [&](int lane) {
    set_offsets(lane);
    const bool words = LAYOUT != TA && (at.koff & 7) != 0 && at.kbeg == 0;
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      const Half ha = half_setup(at.kbeg + s, s, 0);
      const Half hb = half_setup(at.kbeg + s, s, 1);
      if (LAYOUT != TA && s == 0 && words)
        first_words(ha, 0, lane);
      else
#pragma unroll
        for (int i = 0; i < DMA_A; ++i) refill_one(ha, 0, i, lane, true);
      if (LAYOUT == NT && s == 0 && words)
        first_words(hb, 1, lane);
      else
#pragma unroll
        for (int i = 0; i < DMA_B; ++i) refill_one(hb, 1, i, lane, true);
    }
  };
  prologue(opaque_tid() & 63);
  int stores = 0;  // stores of this wave known to have been issued after those loads

  for (;;) {
    // (the lane is read anew for each tile: values derived from it would
    // otherwise be kept through the epilogue)
    const int lane = opaque_tid() & 63;
    const int l16 = lane & 15, lq = lane >> 4;

    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = (f32x4){};
    fence();

    // Fragment read offsets within a stage (gemm_kernel.h).
    int fa[SUB], fb[SUB], fbn[NI];
    [[maybe_unused]] int fan[MI];
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      fa[s] = (wm * WTM + l16) * 128 + (((4 * s + lq) ^ swz_k(l16)) << 4);
      fb[s] = (wn * WTN + l16) * 128 + (((4 * s + lq) ^ swz_k(l16)) << 4);
    }
    {
      const int klane = 8 * lq + (l16 >> 2);
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fbn[j] = klane * (2 * TN) +
                 (((wn * (WTN / 8) + 2 * j + ((lane & 3) >> 1)) ^ swz_rows<TN>(klane)) << 4) +
                 (lane & 1) * 8;
      if constexpr (LAYOUT == TA) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
          fan[i] = klane * (2 * TM) +
                   (((wm * (WTM / 8) + 2 * i + ((lane & 3) >> 1)) ^ swz_rows<TM>(klane)) << 4) +
                   (lane & 1) * 8;
      }
    }
    struct Frags {
      u32x4 a[MI];
      u32x4 b[NI];
    };
    constexpr int A_READS = LAYOUT == TA ? 2 * MI : MI;
    constexpr int READS = A_READS + (LAYOUT == NT ? NI : 2 * NI);
    auto read_item = [&](int es, int ls, int s, Frags& F, int f) {
      const char* abase = smem + (EARLY == 0 ? es * A_BYTES : RING2 + ls * A_BYTES);
      const char* bbase = smem + (EARLY == 1 ? es * B_BYTES : RING2 + ls * B_BYTES);
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
    auto share = [](int q, int steps, int total, auto&& item) {
#pragma unroll
      for (int f = (q * total) / steps; f < ((q + 1) * total) / steps; ++f) item(f);
    };
    auto mfma_pair = [&](const Frags& F, int q) {
#pragma unroll
      for (int t = 2 * q; t < 2 * q + 2; ++t) {
        const int j = t / MI, i = (j & 1) ? MI - 1 - t % MI : t % MI;
        mfma16<T>(acc[i][j], F.b[j], F.a[i]);
      }
    };

    // Column sums of A: a lane adds the eight k that it holds of each A
    // fragment.  All tiles of a tile row read the same A, so they share the
    // K steps: step ks is added by wave column ks mod (2 tiles_n) of the
    // row's 2 tiles_n (two to a tile), between the substeps, where both
    // substeps' fragments are at hand.  (One v_dot2c per fragment word in
    // every tile and step took 8 to 12% of 5120 x 8192 x 8192; a branch per
    // step costs nothing measurable.)  Short K: the first tile of the row
    // takes all steps, its two wave columns by turns, and needs no second
    // kernel.
    [[maybe_unused]] float cs[MI];
    [[maybe_unused]] int sum_at = 0, sum_step = 2;
    [[maybe_unused]] const bool direct = SUMS && p.colsum_ws == nullptr;
    if constexpr (SUMS) {
#pragma unroll
      for (int i = 0; i < MI; ++i) cs[i] = 0.0f;
      if (direct) {
        sum_at = at.tn == 0 ? wn : at.kend;
      } else {
        sum_step = 2 * p.tiles_n;
        sum_at = at.kbeg + (2 * at.tn + wn + sum_step - at.kbeg % sum_step) % sum_step;
      }
    }

    // Stage 0 has landed; the loads of the stages after it, and the last
    // tile's stores behind them, may still be in flight.
    constexpr int LATER = (AHEAD - 1) * (DMA_A + DMA_B), STORES = WTM * WTN / 512;
    static_assert(LATER + STORES <= 63, "the wait's counter has six bits");
    if (stores)
      wait_vm_barrier<LATER + STORES>();
    else
      wait_vm_barrier<LATER>();
    Frags F0, F1;
#pragma unroll
    for (int f = 0; f < READS; ++f) {
      read_item(0, 0, 0, F0, f);
      fence();
    }

    // The K loop of gemm_kernel.h, AHEAD stages deep: entering step ks, stage
    // ks has landed, the AHEAD - 1 after it are in flight, F0 holds substep 0.
    // Substep 0 loads stage ks + AHEAD's early tile into the slot of stage ks
    // - 1; after the barrier in substep 1 (stage ks + 1 landed, every wave
    // done with stage ks) its other tile goes into the slot of stage ks.
    int es = 0;  // early-ring slot of stage ks
    for (int ks = at.kbeg; ks < at.kend; ++ks) {
      const int ls = (ks - at.kbeg) & (AHEAD - 1);       // other-ring slot of stage ks
      const int es1 = es == AHEAD ? 0 : es + 1;          // early-ring slot of stage ks + 1
      const int es_load = es == 0 ? AHEAD : es - 1;      // and of stage ks + AHEAD
      Half he;
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        share(q, PAIRS, READS, [&](int f) { read_item(es, ls, 1, F1, f); });
        mfma_pair(F0, q);
        fence();
        if (q == 0) he = half_setup(ks + AHEAD, es_load, EARLY);
        share(q, PAIRS, DMA_E, [&](int i) { refill_one(he, EARLY, i, lane, false); });
      }
      if constexpr (SUMS) {
        if (ks == sum_at) {
          sum_at += sum_step;
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
                [&](int f) { read_item(es1, (ls + 1) & (AHEAD - 1), 0, F0, f); });
        mfma_pair(F1, q);
        fence();
        if (q >= BAR_PAIR)
          share(q - BAR_PAIR, PAIRS - BAR_PAIR, DMA_L,
                [&](int i) { refill_one(hl, 1 - EARLY, i, lane, false); });
      }
      es = es1;
    }

    wait_vm_barrier<0>();  // every wave is done with the rings
    // wait states between the last MFMAs and the first reads of their results
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    fence();

    if constexpr (SUMS) {
      // the four lane groups' sums of each column, added in a fixed order;
      // column_sums adds those of the tile row's wave columns
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        cs[i] += __shfl_xor(cs[i], 16);
        cs[i] += __shfl_xor(cs[i], 32);
      }
      if (!direct) {
        float* w = p.colsum_ws + ((size_t)at.task * 2 + wn) * TM + wm * WTM;
#pragma unroll
        for (int i = 0; i < MI; ++i)
          if (lq == 0) w[16 * i + l16] = cs[i];
      } else if (at.tn == 0) {
        // the second wave column's sums to the first, through the place in
        // LDS where that wave alone will stage its outputs
        float* x = (float*)(smem + STAGE_AT + 2 * wm * (STAGING / WAVES));
        if (wn == 1 && lq == 0)
#pragma unroll
          for (int i = 0; i < MI; ++i) x[16 * i + l16] = cs[i];
        __syncthreads();
        if (wn == 0 && lq == 0)
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const int m = at.m0 + wm * WTM + 16 * i + l16;
            if (m < at.M)
              p.colsum[(int64_t)at.group * p.M + m] = (uint16_t)pack2<T>(cs[i] + x[16 * i + l16], 0.0f);
          }
      }
    }

    // The next tile's first loads: for A.T @ B ahead of this one's outputs (32
    // groups of 128 rows, 2048 x 2048, 82 -> 80 us; 16 of 1024, 4096 x 4096,
    // 552 -> 545).  With an epilogue after them: its own loads would queue
    // behind them (16 groups of 1024 rows, N = K = 4096, 430 us, 436 ahead).
    constexpr bool FIRST = LAYOUT == TA;
    const TileAt out = at;
    task += stride;
    const bool last = task >= num_tasks;
    if (FIRST && !last) {
      at = locate(task);
      prologue(lane);
    }
    char* stg = smem + STAGE_AT + wave * (STAGING / WAVES);
    const int col0 = out.n0 + wn * WTN, row0 = out.m0 + wm * WTM;
    // interior tiles issue every store of a wave, STORES of them, after those
    // loads
    const bool interior = !out.part && out.vm == TM && out.vn == TN;
    stores = FIRST && interior;

    if constexpr (EPI) {
      // Per 16-row block the wave's FP32 accumulators are staged in LDS (rows
      // of CHF 16-byte chunks), so that each lane gets eight consecutive
      // columns of a row and reads the residual or Z, and writes Z and D, in
      // 16-byte accesses.  (Staged in 16 bits, as below, the residual could
      // only be added after a first rounding.)  Chunk c of row r is stored at
      // c ^ (c >> 3 & 1) ^ (r & 7): the writes (one chunk of eight rows) and
      // the reads (every other chunk of a row) both touch distinct banks.
      // The loop over the blocks is not unrolled: the code of eight
      // activations and slopes stays small enough for the instruction cache
      // beside the K loop.  A pass reads the next one's residual or Z from
      // memory before it computes, and where a wave has its SIMD to itself
      // (nothing else would cover the latency) the next one's values from LDS
      // too: 4096^3 without an activation 103 -> 97 us; with two workgroups
      // per CU the registers that takes cost more (48 ragged groups, 53 us
      // against 56).
      constexpr int CH = WTN / 8;    // lanes per staged row
      constexpr int CHF = WTN / 4;   // 16-byte chunks per staged row
      constexpr int RPI = 64 / CH;   // rows per wave instruction
      constexpr int R = 16 / RPI;    // row instructions per pass
      constexpr bool PIPE = per_cu<SPLIT, TN, TM>() == 1;
      const Epilogue& ep = p.e;
      const int cc = lane % CH, rl = lane / CH;
      const int col = col0 + cc * 8;
      uint32_t bias[4] = {0u, 0u, 0u, 0u};
      if (!ep.grad && ep.bias != nullptr && col < p.N)
        load_row<4>(ep.bias + out.group * ep.bias_stride, col, p.N, bias);
      // the operand each output needs: the residual, or the gradient's Z
      const uint16_t* side = ep.grad ? ep.z : ep.res;
      const int64_t ld_side = ep.grad ? ep.ldz : ep.ldr;
      // (int8: the columns' scales, and with the side values the rows')
      [[maybe_unused]] float sb[8] = {};
      if constexpr (is_i8<T>) {
        if (!out.part) load_scales(p.s.b + out.group * p.s.b_stride, col, p.N, sb);
      }
      auto fetch = [&](int pass, uint32_t(&w)[R][4], [[maybe_unused]] float(&sa)[R]) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int row = row0 + pass * 16 + t * RPI + rl;
          if constexpr (is_i8<T>) sa[t] = !out.part && row < out.M ? p.s.a[row] : 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) w[t][k] = 0u;
          if (side != nullptr && !out.part && row < out.M && col < p.N)
            load_row<4>(side + row * ld_side, col, p.N, w[t]);
        }
      };
      auto stage = [&](int i) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int c = 4 * j + lq;
          *(f32x4*)(stg + ((l16 * CHF + (c ^ ((c >> 3) & 1) ^ (l16 & 7))) << 4)) = acc[i][j];
        }
      };
      auto read_staged = [&](float(&v)[R][8]) {
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int r = t * RPI + rl;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 2 * cc + h;
            const f32x4 x = *(const f32x4*)(stg + ((r * CHF + (c ^ ((c >> 3) & 1) ^ (r & 7))) << 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[t][4 * h + k] = x[k];
          }
        }
      };
      uint32_t w[R][4], w_next[R][4] = {};
      float sa[R] = {}, sa_next[R] = {};
      fetch(0, w, sa);
      stage(0);
      // Loads are waited for on every path (the empty asm uses their
      // results): one that the compiler believes pending when the next tile's
      // K loop begins makes it wait for all loads inside that loop.
      asm volatile("" : "+v"(bias[0]), "+v"(bias[1]), "+v"(bias[2]), "+v"(bias[3]));
#pragma unroll
      for (int t = 0; t < R; ++t)
        asm volatile("" : "+v"(w[t][0]), "+v"(w[t][1]), "+v"(w[t][2]), "+v"(w[t][3]));
      if constexpr (is_i8<T>) {
#pragma unroll
        for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(sb[k]));
#pragma unroll
        for (int t = 0; t < R; ++t) asm volatile("" : "+v"(sa[t]));
      }
      float v[R][8];
      [[maybe_unused]] float v_next[R][8];
      if constexpr (PIPE) read_staged(v);
#pragma unroll 1
      for (int pass = 0; pass < MI; ++pass) {
        // (a wave's LDS accesses complete in order: the next block's writes
        // follow the reads of this one's values)
        switch (PIPE ? pass + 1 : pass) {  // the block to stage now
          case 1: stage(1); break;
          case 2: stage(2); break;
          case 3: stage(3); break;
          case 4: if constexpr (MI > 4) stage(4); break;
          case 5: if constexpr (MI > 4) stage(5); break;
          case 6: if constexpr (MI > 4) stage(6); break;
          case 7: if constexpr (MI > 4) stage(7); break;
          default: break;
        }
        if (pass + 1 < MI) {
          fetch(pass + 1, w_next, sa_next);
          if constexpr (PIPE) read_staged(v_next);
        }
        if constexpr (!PIPE) read_staged(v);
        if (out.part) {
          // the part's FP32 partial tile, row-major TM x TN (elements outside
          // D are skipped: nothing reads them)
          float* ws = p.ws + (size_t)out.part_index * (TM * TN) + wn * WTN + cc * 8;
#pragma unroll
          for (int t = 0; t < R; ++t) {
            const int r = wm * WTM + pass * 16 + t * RPI + rl;
            if (out.m0 + r < out.M && col < p.N) {
              *(f32x4*)(ws + r * TN) = (f32x4){v[t][0], v[t][1], v[t][2], v[t][3]};
              *(f32x4*)(ws + r * TN + 4) = (f32x4){v[t][4], v[t][5], v[t][6], v[t][7]};
            }
          }
        } else if (!is_i8<T> && ep.grad) {
          if constexpr (!is_i8<T>) apply_slope<T>(ep.act, v, w);
        } else {
          if constexpr (is_i8<T>) {
#pragma unroll
            for (int t = 0; t < R; ++t)
#pragma unroll
              for (int k = 0; k < 8; ++k) v[t][k] = scaled(__builtin_bit_cast(int, v[t][k]), sa[t], sb[k]);
          }
#pragma unroll
          for (int t = 0; t < R; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[t][k] += unpack<O>(bias[k >> 1], k & 1);
          if (ep.z != nullptr) {
#pragma unroll
            for (int t = 0; t < R; ++t) {
              const int row = row0 + pass * 16 + t * RPI + rl;
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = pack2<O>(v[t][2 * k], v[t][2 * k + 1]);
              if (row < out.M && col < p.N)
                store_row<4>(ep.z + (int64_t)row * ep.ldz, col, p.N, o);
            }
          }
          apply_act(ep.act, v);
          if (ep.res != nullptr) {
#pragma unroll
            for (int t = 0; t < R; ++t)
#pragma unroll
              for (int k = 0; k < 8; ++k) v[t][k] += unpack<O>(w[t][k >> 1], k & 1);
          }
        }
#pragma unroll
        for (int t = 0; t < R; ++t) {
          asm volatile("" : "+v"(w_next[t][0]), "+v"(w_next[t][1]), "+v"(w_next[t][2]),
                       "+v"(w_next[t][3]));
          if constexpr (is_i8<T>) {
            asm volatile("" : "+v"(sa_next[t]));
            sa[t] = sa_next[t];
          }
        }
#pragma unroll
        for (int t = 0; t < R; ++t) {
          const int row = row0 + pass * 16 + t * RPI + rl;
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = pack2<O>(v[t][2 * k], v[t][2 * k + 1]);
          if (!out.part && row < out.M && col < p.N)
            store_row<4>(out.D + (int64_t)row * p.ldd, col, p.N, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) w[t][k] = w_next[t][k];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if constexpr (PIPE) v[t][k] = v_next[t][k];
        }
      }
    } else if (out.part) {
      // FP32 partial tile: lane holds row l16 of each 16-row block and columns
      // j*16 + 4*lq .. +3; blocks wholly outside D are skipped
      float* w = p.ws + (size_t)out.part_index * (TM * TN) + (size_t)(wm * WTM + l16) * TN +
                 wn * WTN + 4 * lq;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (wm * WTM + i * 16 >= out.vm) break;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (wn * WTN + j * 16 >= out.vn) break;
          *(f32x4*)(w + i * 16 * TN + j * 16) = acc[i][j];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // Per 32-row band: round, stage in LDS in 16 bits (rows of CH 16-byte
      // chunks, swizzled by row), store 16-byte row chunks; each phase issued
      // whole before the next.
      constexpr int CH = WTN / 8;     // 16-byte chunks per staged row
      constexpr int RPI = 64 / CH;    // rows per wave instruction
      constexpr int NR = 32 / RPI;
#pragma unroll
      for (int band = 0; band < MI / 2; ++band) {
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
          const int r = half * 16 + l16;
#pragma unroll
          for (int j = 0; j < NI; ++j) {
            const int c = 2 * j + (lq >> 1);
            *(u32x2*)(stg + r * (CH * 16) + ((c ^ (r & (CH - 1))) << 4) + (lq & 1) * 8) = v[half][j];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        const int cc = lane % CH, rl = lane / CH;
        const int col = col0 + cc * 8;
        u32x4 o[NR];
#pragma unroll
        for (int t = 0; t < NR; ++t) {
          const int r = t * RPI + rl;
          o[t] = *(const u32x4*)(stg + r * (CH * 16) + ((cc ^ (r & (CH - 1))) << 4));
        }
        __builtin_amdgcn_sched_barrier(0);
        uint16_t* dst = out.D + (int64_t)(row0 + band * 32 + rl) * p.ldd;
        if (interior) {
#pragma unroll
          for (int t = 0; t < NR; ++t)
            __builtin_nontemporal_store(o[t], (u32x4_any*)(dst + (int64_t)t * RPI * p.ldd + col));
        } else {
#pragma unroll
          for (int t = 0; t < NR; ++t) {
            const uint32_t words[4] = {o[t][0], o[t][1], o[t][2], o[t][3]};
            if (row0 + band * 32 + t * RPI + rl < out.M && col < p.N)
              store_row<4>(dst + (int64_t)t * RPI * p.ldd, col, p.N, words);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (last) return;
    if (!FIRST) {
      at = locate(task);
      prologue(lane);
    }
  }
}

}  // namespace dg
