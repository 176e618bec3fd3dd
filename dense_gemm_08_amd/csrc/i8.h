// i8.h -- int8 operands of a layer's products on the MI355X (gfx950): the type
// that selects them in the kernels' templates, their MFMA, and the scales that
// turn the sums of whole numbers into values.
//
//   P = sum_k A[i][k] B[j][k]           in 32-bit integers, exactly
//   Z = P sa[i] sb[j] + bias            in FP32, then as for 16-bit operands
//
// A row of K int8 values is moved and staged as a row of K / 2 16-bit ones:
// v_mfma_i32_16x16x64_i8 takes 16 bytes of a row from each lane where
// v_mfma_f32_16x16x32 takes eight 16-bit values, its result has the same
// layout, and it takes the same time for twice the products.  So the loads, the
// rings, the schedule and the tile choice are those of the 16-bit products with
// half the K.
//
// Measured on the MI355X: 8192 x 5120 x 17408 562 us, 2600 TOP/s (the 16-bit
// product 1104 us; the board's power limits both, MFMA busy 0.76); 3000 x 5000 x
// 4000 with GELU and Z 67 us, of which the K steps take 43 and the one round's
// epilogue, 60 MB written by all CUs at once, most of the rest.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"

namespace dg {

template <typename O>
struct I8 {
  typedef O output;
};
template <typename T>
constexpr bool is_i8 = false;
template <typename O>
constexpr bool is_i8<I8<O>> = true;

template <typename T>
struct OutputOf {
  typedef T type;
};
template <typename O>
struct OutputOf<I8<O>> {
  typedef O type;
};
template <typename T>
using output_of = typename OutputOf<T>::type;

struct I8Scales {
  const float* a;    // one per row of A
  const float* b;    // one per row of B
  int64_t b_stride;  // elements between the groups' scales of B
};

// (the wait states are the kernels', as for the other MFMAs of cdna_ops.h)
template <>
__device__ __forceinline__ void mfma16<I8<_Float16>>(f32x4& c, u32x4 a, u32x4 b) {
  asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
template <>
__device__ __forceinline__ void mfma16<I8<__bf16>>(f32x4& c, u32x4 a, u32x4 b) {
  asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// A sum times its two scales.  The products are not fused with the addition that
// follows: every kernel rounds alike, so a row's results do not depend on the
// tiles that a call takes.
__device__ __forceinline__ float scaled(int sum, float sa, float sb) {
#pragma clang fp contract(off)
  const float x = (float)sum * sa;
  return x * sb;
}

// C scales of consecutive columns from column col of `cols` on; zeros past it.
template <int C>
__device__ __forceinline__ void load_scales(const float* s, int col, int cols, float (&v)[C]) {
  typedef f32x4 f32x4_any __attribute__((aligned(4)));
#pragma unroll
  for (int c = 0; c < C; c += 4) {
    if (col + c + 4 <= cols) {
      const f32x4 x = *(const f32x4_any*)(s + col + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c + k] = x[k];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[c + k] = col + c + k < cols ? s[col + c + k] : 0.0f;
    }
  }
}

}  // namespace dg
