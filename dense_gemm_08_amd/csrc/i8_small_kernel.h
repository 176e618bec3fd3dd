// i8_small_kernel.h -- the int8 product for small outputs on the MI355X
// (gfx950): gemm_small_kernel.h's decomposition, whose comments explain it
// (16-row or 32-row tiles of 16 or 32 columns, a workgroup each; eight waves
// that split K; a ring of LDS-DMA loads per wave, no barrier in the K loop; the
// waves' sums added through LDS), on v_mfma_i32_16x16x64_i8.
//
// What differs: a chunk is 128 int8 values of each row; the sums are whole
// numbers, so their order changes nothing; and rows of any K are read in place
// where they begin at 4-byte addresses: the bytes behind K in a row's last
// 16-byte piece, the next row's, are cleared in A's fragments alone, as 0 times
// any int8 value is 0.
//
// Bound by memory: 1 x 16384 x 4096 13.2 us (5.1 TB/s, operands from HBM), 8 x 8192
// x 8192 12.4, 1 x 4096 x 4096 5.1 (a launch's latency).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"
#include "epilogue.h"
#include "groups.h"
#include "i8.h"
#include "tile_config.h"
#include "tile_sched.h"

namespace dg {

struct SmallI8Params {
  const int8_t* A;
  const int8_t* B;
  uint16_t* D;
  int M, N, K;
  int lda, ldb;          // bytes
  int ldd;
  int tiles_m, tiles_n;  // tiles of the launch's shape
  int num_xcds;
  Epilogue e;
  I8Scales s;
  Groups g;              // (stride in bytes)
};

template <typename O, int TMB, int TNB, bool GROUP>
__global__ __launch_bounds__(SMALL_THREADS) void gemm_small_i8(SmallI8Params p) {
  constexpr int RING = 2;
  constexpr int TR = SMALL_TILE * TMB, TC = SMALL_TILE * TNB;
  constexpr int SLOT = (TR + TC) * 128;
  constexpr int BLOCKS = TMB * TNB;
  constexpr int LOADS = 2 * (TMB + TNB);
  static_assert(BLOCKS <= SMALL_WAVES, "one wave per block in the final sum");
  static_assert(SMALL_WAVES * BLOCKS * 64 * 16 <= SMALL_WAVES * RING * SLOT,
                "the waves' partial blocks fit in the rings they replace");
  __shared__ __attribute__((aligned(1024))) char ring[SMALL_WAVES * RING * SLOT];

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lane = (int)threadIdx.x & 63;
  const int l16 = lane & 15, lq = lane >> 4;
  int tile, tiles_m = p.tiles_m, row0 = 0, M = p.M;
  const int8_t* gB = p.B;
  [[maybe_unused]] int group = 0;
  if constexpr (GROUP) {
    GroupMap<1> map;
    map.count(p.g, TR, p.tiles_n);
    if ((int)blockIdx.x >= map.total) return;
    GroupTile t;
    map.find(p.g, xcd_slot((int)blockIdx.x, map.total, p.num_xcds), TR, p.tiles_n, &t);
    tile = t.tile;
    group = t.group;
    row0 = t.beg;
    M = t.end;
    tiles_m = (M - row0 + TR - 1) / TR;
    gB += group * p.g.stride;
  } else {
    tile = xcd_slot((int)blockIdx.x, (int)gridDim.x, p.num_xcds);
  }
  const int tm = tile % tiles_m, tn = tile / tiles_m;
  const int m0 = row0 + tm * TR, n0 = tn * TC;
  const int vm = min(TR, M - m0), vn = min(TC, p.N - n0);

  // (a range ends with the word that holds the last value: rows begin at whole
  // words, so it is one the matrix reaches into)
  const uint32_t K4 = (uint32_t)(p.K + 3) & ~3u;
  const i32x4 ra = make_rsrc((uint64_t)(uintptr_t)(p.A + (int64_t)m0 * p.lda),
                             (uint32_t)((vm - 1) * p.lda) + K4);
  const i32x4 rb = make_rsrc((uint64_t)(uintptr_t)(gB + (int64_t)n0 * p.ldb),
                             (uint32_t)((vn - 1) * p.ldb) + K4);
  uint32_t aoff[2 * TMB], boff[2 * TNB];
  int kca[2 * TMB], kcb[2 * TNB];
#pragma unroll
  for (int i = 0; i < 2 * TMB; ++i) {
    const int r = 8 * i + (lane >> 3);
    kca[i] = (lane & 7) ^ swz_k(r);
    aoff[i] = r < vm ? (uint32_t)(r * p.lda + kca[i] * 16) : OOB;
  }
#pragma unroll
  for (int j = 0; j < 2 * TNB; ++j) {
    const int r = 8 * j + (lane >> 3);
    kcb[j] = (lane & 7) ^ swz_k(r);
    boff[j] = r < vn ? (uint32_t)(r * p.ldb + kcb[j] * 16) : OOB;
  }
  const uint32_t wring = lds_addr(ring) + wave * (RING * SLOT);
  // chunk t of this wave (K chunk wave + 8 t) into ring slot t % RING; pieces at
  // or past K read zeros
  auto issue = [&](int t) {
    const int c = wave + SMALL_WAVES * t;
    const uint32_t base = wring + (t % RING) * SLOT;
#pragma unroll
    for (int i = 0; i < 2 * TMB; ++i)
      dma16_at(ra, c * 128 + kca[i] * 16 < p.K ? aoff[i] + c * 128 : OOB, base, i * 1024);
#pragma unroll
    for (int j = 0; j < 2 * TNB; ++j)
      dma16_at(rb, c * 128 + kcb[j] * 16 < p.K ? boff[j] + c * 128 : OOB, base, TR * 128 + j * 1024);
  };
  const int fr0 = l16 * 128 + ((lq ^ swz_k(l16)) << 4);
  const int fr1 = l16 * 128 + (((4 + lq) ^ swz_k(l16)) << 4);
  // a fragment's bytes k .. k + 15 without those at or past K
  auto clip = [&](u32x4 x, int k) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int left = p.K - k - 4 * w;  // bytes of the word that count
      x[w] &= left >= 4 ? 0xffffffffu : left > 0 ? (1u << (8 * left)) - 1 : 0u;
    }
    return x;
  };

  const int chunks = (p.K + 127) / 128;
  const int per_wave = (chunks + SMALL_WAVES - 1) / SMALL_WAVES;
  i32x4 acc0[TMB][TNB], acc1[TMB][TNB];
#pragma unroll
  for (int i = 0; i < TMB; ++i)
#pragma unroll
    for (int j = 0; j < TNB; ++j) acc0[i][j] = acc1[i][j] = i32x4{0, 0, 0, 0};
  if (per_wave > 0) {  // (K = 0: no loads at all)
    for (int t = 0; t < RING; ++t) issue(t);
    for (int t = 0; t < per_wave; ++t) {
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LOADS * (RING - 1)) : "memory");
      const char* slot = ring + (wave * RING + t % RING) * SLOT;
      const int k0 = (wave + SMALL_WAVES * t) * 128 + 16 * lq;
      u32x4 a0[TMB], a1[TMB], b0[TNB], b1[TNB];
#pragma unroll
      for (int i = 0; i < TMB; ++i) {
        a0[i] = *(const u32x4*)(slot + i * 2048 + fr0);
        a1[i] = *(const u32x4*)(slot + i * 2048 + fr1);
      }
      if ((wave + SMALL_WAVES * t) * 128 + 128 > p.K) {
#pragma unroll
        for (int i = 0; i < TMB; ++i) {
          a0[i] = clip(a0[i], k0);
          a1[i] = clip(a1[i], k0 + 64);
        }
      }
#pragma unroll
      for (int j = 0; j < TNB; ++j) {
        b0[j] = *(const u32x4*)(slot + (TR + SMALL_TILE * j) * 128 + fr0);
        b1[j] = *(const u32x4*)(slot + (TR + SMALL_TILE * j) * 128 + fr1);
      }
#pragma unroll
      for (int i = 0; i < TMB; ++i)
#pragma unroll
        for (int j = 0; j < TNB; ++j) {
          acc0[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b0[j]),
                                                             __builtin_bit_cast(i32x4, a0[i]),
                                                             acc0[i][j], 0, 0, 0);
          acc1[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b1[j]),
                                                             __builtin_bit_cast(i32x4, a1[i]),
                                                             acc1[i][j], 0, 0, 0);
        }
      // the slot's reads are done (the MFMAs took their data): refill it
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
      issue(t + RING);
    }
    // no LDS-DMA write may land after the wave ends
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  }

  __syncthreads();
  i32x4(*part)[BLOCKS][64] = reinterpret_cast<i32x4(*)[BLOCKS][64]>(ring);
#pragma unroll
  for (int i = 0; i < TMB; ++i)
#pragma unroll
    for (int j = 0; j < TNB; ++j) part[wave][i * TNB + j][lane] = acc0[i][j] + acc1[i][j];
  __syncthreads();
  if (wave >= BLOCKS) return;
  i32x4 s = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < SMALL_WAVES; ++w) s += part[w][wave][lane];
  const int row = m0 + SMALL_TILE * (wave / TNB) + l16;
  const int col = n0 + SMALL_TILE * (wave % TNB) + 4 * lq;
  if (row >= M || col >= p.N) return;
  float sb[4], x[1][4];
  load_scales(p.s.b + group * p.s.b_stride, col, p.N, sb);
  const float sa = p.s.a[row];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[0][k] = scaled(s[k], sa, sb[k]);
  finish_row<O>(p.e, group, row, col, p.N, x);
  const uint32_t o[2] = {pack2<O>(x[0][0], x[0][1]), pack2<O>(x[0][2], x[0][3])};
  store_row<2>(p.D + (int64_t)row * p.ldd, col, p.N, o);
}

// The parts of split tiles (layer_kernel.h's SPLIT kernels), summed as whole
// numbers, then scaled and finished: split_reduce.h's map of threads to
// elements, eight consecutive columns of a row each.
struct I8ReduceParams {
  const int32_t* ws;
  uint16_t* D;
  int M, N, ldd;
  int tiles_m, tiles_n, group_m;
  int full_tasks, splits, tiles;
  Epilogue e;
  I8Scales s;
};
constexpr int I8_REDUCE_THREADS = 64;
template <typename O, int TN, int TM>
__global__ __launch_bounds__(I8_REDUCE_THREADS) void split_reduce_i8(I8ReduceParams p) {
  constexpr int TPR = TN / 8, RPW = I8_REDUCE_THREADS / TPR, WPT = TM / RPW;
  const int st = blockIdx.x / WPT;
  int tm, tn;
  tile_of_task(p.full_tasks + st, p.tiles_m, p.tiles_n, p.group_m, &tm, &tn);
  const int r = (blockIdx.x % WPT) * RPW + (int)threadIdx.x / TPR;
  const int c = ((int)threadIdx.x % TPR) * 8;
  const int row = tm * TM + r, col = tn * TN + c;
  if (row >= p.M || col >= p.N) return;
  const int32_t* w = p.ws + (size_t)st * (TM * TN) + (size_t)r * TN + c;
  const size_t stride = (size_t)p.tiles * (TM * TN);
  i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
#pragma unroll 8
  for (int k = 0; k < p.splits; ++k) {
    lo += *(const i32x4*)(w + k * stride);
    hi += *(const i32x4*)(w + k * stride + 4);
  }
  float sb[8], x[1][8];
  load_scales(p.s.b, col, p.N, sb);
  const float sa = p.s.a[row];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[0][k] = scaled(k < 4 ? lo[k & 3] : hi[k & 3], sa, sb[k]);
  finish_row<O>(p.e, 0, row, col, p.N, x);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = pack2<O>(x[0][2 * k], x[0][2 * k + 1]);
  store_row<4>(p.D + (int64_t)row * p.ldd, col, p.N, o);
}

// Copies of operands whose rows the kernels cannot read in place: `count`
// matrices of rows x cols bytes, at any address and distance, into dense ones
// whose rows are dcols bytes (a multiple of 16), zeros behind cols.
struct I8RepackJob {
  const int8_t* src;
  int8_t* dst;
  int64_t count, rows, cols, ld, stride, dcols;
  int64_t blocks;
  int lanes;  // lanes per row, a power of two up to 256
};
typedef u32x4 u32x4_byte __attribute__((aligned(1)));
[[maybe_unused]] static __global__ __launch_bounds__(256) void repack_i8(I8RepackJob a, I8RepackJob b) {
  const bool first = blockIdx.x < a.blocks;
  const I8RepackJob& j = first ? a : b;
  const int64_t block = first ? blockIdx.x : blockIdx.x - a.blocks;
  const int shift = __builtin_ctz(j.lanes), lane = (int)threadIdx.x & (j.lanes - 1);
  const int per = 256 >> shift;
  const int64_t total = j.count * j.rows;
  for (int64_t r = block * per + ((int)threadIdx.x >> shift); r < total; r += j.blocks * per) {
    const int64_t g = j.count > 1 ? r / j.rows : 0;
    const int8_t* src = j.src + g * j.stride + (r - g * j.rows) * j.ld;
    for (int64_t c = lane * 16; c < j.dcols; c += j.lanes * 16) {
      u32x4 x = {0, 0, 0, 0};
      if (c + 16 <= j.cols) {
        x = *(const u32x4_byte*)(src + c);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c + k < j.cols) x[k >> 2] |= (uint32_t)(uint8_t)src[c + k] << (8 * (k & 3));
      }
      *(u32x4*)(j.dst + r * j.dcols + c) = x;
    }
  }
}

}  // namespace dg
