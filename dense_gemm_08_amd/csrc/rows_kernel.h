// rows_kernel.h -- what happens to rows around an expert layer's products on
// the MI355X (gfx950): rows quantised to int8 with a scale each (gathered by
// token where they are sent to experts), and the experts' rows added up per
// token, with the gradients of that sum.
//
// All of them move every element once, and memory bounds them: a lane takes
// eight neighbouring 16-bit elements at a time (16-byte accesses at any
// alignment) and a row is shared by 16, 64, 256 or 1024 lanes, by its length
// and by the number of rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"
#include "epilogue.h"
#include "lanes.h"

namespace dg {

constexpr int ROW_CHUNKS = 8;  // pieces of eight elements that a lane holds of a row

// The threads of a block that shares a row among W lanes, and the rows of such
// a block.
template <int W>
constexpr int row_threads() { return W < 256 ? 256 : W; }
template <int W>
constexpr int rows_per_block() { return row_threads<W>() / W; }

// body(row) for the rows of this block, the same number of times in every lane
// (a row at or past count: nothing to do but to take part).  A launch holds
// fewer than 2^32 threads: more rows than these can have are taken in turns.
template <int W, typename Body>
__device__ __forceinline__ void for_rows(int64_t count, Body&& body) {
  constexpr int per = rows_per_block<W>();
  for (int64_t row = (int64_t)blockIdx.x * per; row < count; row += (int64_t)gridDim.x * per)
    body(row + (int)threadIdx.x / W);
}

// x of the W lanes that share a row, combined by op; scratch: one X per wave.
template <int W, typename X, typename Op>
__device__ __forceinline__ X reduce_row(X x, X* scratch, Op&& op) {
  x = reduce_lanes<W == 16 ? 16 : 64>(x, op);
  if constexpr (W > 64) {
    const int wave = (int)threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) scratch[wave] = x;
    __syncthreads();
    x = scratch[0];
#pragma unroll
    for (int w = 1; w < W / 64; ++w) x = op(x, scratch[w]);
    __syncthreads();
  }
  return x;
}

// ---- int8 ------------------------------------------------------------------

struct QuantizeParams {
  const uint16_t* X;
  const int32_t* rows;  // the row of X that row i of Q is made of, or null: i
  int8_t* Q;
  float* S;
  int64_t ldx, ldq;
  int64_t count;   // rows of Q
  int64_t x_rows;  // rows of X
  int K;
};

typedef u32x2 u32x2_byte __attribute__((aligned(1)));

// Q[i][k] = round(127 x / m), half-way cases to even, S[i] = m / 127 with m the
// largest |x| of the row.  The quotient is formed so that no rounding of it
// moves a value across a half-way point: x and m have at most 11 significant
// bits, so 127 x / m is either k + 1/2 exactly or at least 2^-19 of its size
// away from it; as x times 127 / m in two floats it is rounded once from a value
// within 2^-47 of it, which gives k + 1/2 itself wherever that is the quotient.
// m of a row: the largest of the 16-bit patterns without their sign, which are
// ordered as the sizes they stand for, infinities and NaNs last, two at a time.
// A row that holds one of those gets the scale NaN (and zeros), a row of zeros
// the scale 0, and a row whose index leads to no row of X is zeros with scale 0.
// Bound by memory: 16384 rows of 4096 in order 32 us, gathered by token (8192
// tokens twice each, whose second read no longer hits L2) 31.5: 131 MB fetched and
// 69 written.  Rows stay in registers between the maximum and the quotients (up
// to 65536 elements), stores past the caches (32.8 without).
template <typename T, int W>
__device__ __forceinline__ void quantize_row(const QuantizeParams& p, int64_t row, uint32_t* scratch) {
  constexpr int SPAN = W * ROW_CHUNKS * 8;  // elements of a row that the lanes hold
  constexpr uint32_t INF = sizeof(T) == 2 && __is_same(T, _Float16) ? 0x7c00u : 0x7f80u;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const int lane = (int)threadIdx.x & (W - 1);
  const bool live = row < p.count;
  int64_t from = row;
  if (p.rows != nullptr) from = live ? p.rows[row] : -1;
  const bool there = live && from >= 0 && from < p.x_rows;
  const uint16_t* src = p.X + (there ? from * p.ldx : 0);
  const int K = there ? p.K : 0;

  uint32_t v[ROW_CHUNKS][4];
  auto load = [&](int64_t first) {
#pragma unroll
    for (int c = 0; c < ROW_CHUNKS; ++c) {
      const int64_t k = first + (c * W + lane) * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[c][e] = 0u;
      if (k < K) load_row<4>(src, (int)k, K, v[c]);
    }
  };
  u16x2 m = {0, 0};
  // (the last segment is the one held when the loop ends, the only one of a row
  // that fits; a longer row is read twice)
  for (int64_t first = 0; first < p.K; first += SPAN) {
    load(first);
#pragma unroll
    for (int c = 0; c < ROW_CHUNKS; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[c][e] & 0x7fff7fffu));
  }
  const uint32_t top = reduce_row<W>((uint32_t)(m[0] > m[1] ? m[0] : m[1]), scratch,
                                     [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  if (!live) return;
  const bool finite = top < INF;
  const float most = finite ? unpack<T>(top, 0) : 0.0f;
  if (lane == 0) p.S[row] = finite ? most / 127.0f : __builtin_nanf("");
  // Rows whose largest value is far from 1 are brought nearer by a power of two
  // (127 / m and its second part then neither overflow nor vanish; what falls
  // below FP32's smallest is far below m / 254).
  const bool far = most != 0.0f && !(most > 0x1p-64f && most < 0x1p64f);
  const float pull = far ? (most < 1.0f ? 0x1p64f : 0x1p-64f) : 1.0f;
  const float m1 = most > 0.0f ? most * pull : 1.0f;
  const float hi = 127.0f / m1, lo = fmaf(-hi, m1, 127.0f) / m1;  // (the remainder is exact)
  int8_t* dst = p.Q + row * p.ldq;
  for (int64_t first = 0; first < p.K; first += SPAN) {
    if (p.K > SPAN) load(first);
#pragma unroll
    for (int c = 0; c < ROW_CHUNKS; ++c) {
      const int64_t k = first + (c * W + lane) * 8;
      if (k >= p.K) break;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = unpack<T>(v[c][e >> 1], e & 1);
      if (far || !finite) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = finite ? x[e] * pull : 0.0f;
      }
      uint32_t b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = fmaf(x[e], hi, x[e] * lo);
        // (the sum with 1.5 * 2^23 is rounded to a whole number, which its low
        // byte holds)
        b[e] = __builtin_bit_cast(uint32_t, q + 12582912.0f);
      }
      u32x2 o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000c0cu);
        o[h] = lo | hi;
      }
      if (k + 8 <= p.K) {
        __builtin_nontemporal_store(o, (u32x2_byte*)(dst + k));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e < p.K) dst[k + e] = (int8_t)(o[e >> 2] >> ((e & 3) * 8));
      }
    }
  }
}
template <typename T, int W>
__global__ __launch_bounds__(row_threads<W>()) void quantize_rows_i8(QuantizeParams p) {
  __shared__ uint32_t scratch[W > 64 ? W / 64 : 1];
  for_rows<W>(p.count, [&](int64_t row) { quantize_row<T, W>(p, row, scratch); });
}

// ---- the experts' rows, per token ------------------------------------------

struct CombineParams {
  const uint16_t* H;
  const int32_t* places;
  const float* weights;     // or null: 1
  const uint16_t* residual;  // or null
  uint16_t* Y;
  int64_t ldh, ldr, ldy;
  int64_t count;   // tokens
  int64_t h_rows;
  int N, k;
  int lanes;       // lanes per token, a power of two up to 256
};

// Y[t] = sum_j w[t][j] H[places[t][j]] + residual[t], summed in FP32 in the
// order of j and rounded once.  A place outside H adds w times zero (so that a
// weight that is NaN still shows).  Bound by memory: 8192 tokens, two rows of 4096
// each and a residual, 49.5 us (5.4 TB/s), 41 where the operands lie in the
// Infinity Cache; 4096 tokens, eight rows of 2048, 35 (4.8).
template <typename T>
__device__ __forceinline__ void combine_row(const CombineParams& p, int64_t t) {
  const int32_t* places = p.places + t * p.k;
  const float* w = p.weights != nullptr ? p.weights + t * p.k : nullptr;
  const int64_t step = (int64_t)gridDim.y * p.lanes * 8;
  for (int64_t c = ((int64_t)blockIdx.y * p.lanes + ((int)threadIdx.x & (p.lanes - 1))) * 8; c < p.N;
       c += step) {
    const int col = (int)c;
    float s[8] = {};
    uint32_t r[4] = {};
    if (p.residual != nullptr) load_row<4>(p.residual + t * p.ldr, col, p.N, r);
    // (four rows' loads in flight)
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      uint32_t x[4][4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[u][e] = 0u;
        f[u] = 0.0f;
        if (j0 + u < p.k) {
          const int64_t at = places[j0 + u];
          f[u] = w != nullptr ? w[j0 + u] : 1.0f;
          if (at >= 0 && at < p.h_rows) load_row<4>(p.H + at * p.ldh, col, p.N, x[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = fmaf(f[u], unpack<T>(x[u][e >> 1], e & 1), s[e]);
    }
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += unpack<T>(r[e >> 1], e & 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack2<T>(s[2 * e], s[2 * e + 1]);
    store_row<4>(p.Y + t * p.ldy, col, p.N, o);
  }
}
template <typename T>
__global__ __launch_bounds__(256) void combine_rows(CombineParams p) {
  const int shift = __builtin_ctz(p.lanes), per = 256 >> shift;
  for (int64_t t = (int64_t)blockIdx.x * per + ((int)threadIdx.x >> shift); t < p.count;
       t += (int64_t)gridDim.x * per)
    combine_row<T>(p, t);
}

struct CombineGradParams {
  const uint16_t* DY;
  const uint16_t* H;
  const int32_t* places;
  const float* weights;  // or null: 1
  uint16_t* DH;          // or null
  float* dweights;       // or null
  int64_t lddy, ldh, lddh;
  int64_t count, h_rows;
  int N, k;
};

// DH[places[t][j]] = w[t][j] DY[t] and dweights[t][j] = DY[t] . H[places[t][j]],
// the products' sums in FP32 in a fixed order.  W lanes take one choice (t, j);
// those of a token run side by side and share its row of DY in the caches.  (With
// the row in registers over a loop of the token's choices, each choice waits for
// the last one's sum: 4096 tokens, 8 choices of 2048 columns, 78 us, 56 so.)
// 8192 tokens, 2 choices of 4096, 68 us; DH alone, which reads DY only, 42, and
// dweights alone 38.
template <typename T, int W>
__device__ __forceinline__ void combine_choice_grad(const CombineGradParams& p, int64_t choice, float* scratch) {
  constexpr int SPAN = W * ROW_CHUNKS * 8;
  const int lane = (int)threadIdx.x & (W - 1);
  const bool live = choice < p.count * p.k;
  const int64_t t = live ? (uint32_t)choice / (uint32_t)p.k : 0;  // (choices number less than 2^31)
  const int64_t at = live ? p.places[choice] : -1;
  const bool there = at >= 0 && at < p.h_rows;
  const float w = there && p.weights != nullptr ? p.weights[choice] : 1.0f;
  const uint16_t* dy = p.DY + t * p.lddy;
  const uint16_t* h = p.H + (there ? at : 0) * p.ldh;
  uint16_t* dh = p.DH + (there ? at : 0) * p.lddh;
  float s = 0.0f;
  for (int64_t first = 0; there && first < p.N; first += SPAN) {
    uint32_t v[ROW_CHUNKS][4], x[ROW_CHUNKS][4];
#pragma unroll
    for (int c = 0; c < ROW_CHUNKS; ++c) {
      const int64_t col = first + (c * W + lane) * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[c][e] = x[c][e] = 0u;
      if (col < p.N) {
        load_row<4>(dy, (int)col, p.N, v[c]);
        if (p.dweights != nullptr) load_row<4>(h, (int)col, p.N, x[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < ROW_CHUNKS; ++c) {
      const int64_t col = first + (c * W + lane) * 8;
      if (p.DH != nullptr && col < p.N) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack2<T>(w * unpack<T>(v[c][e], 0), w * unpack<T>(v[c][e], 1));
        store_row<4>(dh, (int)col, p.N, o);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        s = fmaf(unpack<T>(v[c][e >> 1], e & 1), unpack<T>(x[c][e >> 1], e & 1), s);
    }
  }
  if (p.dweights == nullptr) return;
  s = reduce_row<W>(s, scratch, [](float a, float b) { return a + b; });
  if (live && lane == 0) p.dweights[choice] = s;
}
template <typename T, int W>
__global__ __launch_bounds__(row_threads<W>()) void combine_rows_grad(CombineGradParams p) {
  __shared__ float scratch[W > 64 ? W / 64 : 1];
  for_rows<W>(p.count * p.k, [&](int64_t choice) { combine_choice_grad<T, W>(p, choice, scratch); });
}

}  // namespace dg
