// epilogue.h -- what a layer's product does to its FP32 accumulators before
// the one rounding to the output type:
//
//   forward    Z = P + bias,  D = act(Z) + residual   (Z stored on request)
//   gradient   D = P * act'(Z)                        (Z read)
//
// with P the accumulated product.  All of it is computed in FP32 from the
// unrounded accumulator; Z and D are each rounded once.  (The gradient's Z is
// the stored, rounded one: the forward pass keeps it at the layer's own
// precision, half the memory of FP32.)
//
// Activations, with s(w) = 1 / (1 + exp(-w)) and F the standard normal
// distribution function:
//   RELU       max(z, 0)                                derivative at 0: 0
//   GELU       z F(z)
//   GELU_TANH  z s(2 u),  u = sqrt(2 / pi) (z + 0.044715 z^3)
//              (0.5 (1 + tanh u) = s(2 u))
//   SILU       z s(z)
// At infinite z they take their limits; NaN gives NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cdna_ops.h"

namespace dg {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct Epilogue {
  const uint16_t* bias;  // N values, or null
  const uint16_t* res;   // residual, or null
  uint16_t* z;           // forward: receives Z, or null; gradient: Z
  int ldr, ldz;
  int64_t bias_stride;   // elements between the groups' biases
  int act;               // Act
  int grad;              // 1: the gradient form
};

// 1 / (1 + exp(-w)).  (exp overflows to infinity for w < -88: the result is
// then 0, its limit.)
__device__ __forceinline__ float logistic(float w) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w * -1.44269504088896341f));
}

// The two tails' factor of the normal distribution: with y = |z| / sqrt(2),
// F(-|z|) = exp(-y^2) q(y), q(y) = erfc(y) exp(y^2) / 2.  q is a polynomial
// in t = 1 / (1 + 0.375 y), fitted here for least relative error over 0 <= y
// <= 14 (1.4e-6, so the negative tail keeps its relative precision down to
// the smallest 16-bit results, where 1 + erf(z / sqrt(2)) would cancel).
__device__ __forceinline__ float normal_tail(float z, float* gauss) {
  const float y = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.375f, y, 1.0f));
  const float e = __builtin_amdgcn_exp2f(y * y * -1.44269504088896341f);
  float q = -0.13092039f;
  q = fmaf(q, t, 0.37347726f);
  q = fmaf(q, t, -0.10964101f);
  q = fmaf(q, t, 0.26908684f);
  q = fmaf(q, t, 0.17187412f);
  q = fmaf(q, t, 0.21471366f);
  q = fmaf(q, t, 0.21141088f);
  *gauss = e;
  return 0.5f * e * t * q;
}

// a * b with 0 where b is 0 (a may be infinite there)
__device__ __forceinline__ float mul_limit(float a, float b) { return b == 0.0f ? 0.0f : a * b; }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // (keeps NaN)
  if constexpr (ACT == ACT_GELU) {
    float e;
    const float q = normal_tail(z, &e);
    return mul_limit(z, z < 0.0f ? q : 1.0f - q);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    const float w = 1.59576912160573071f * z * fmaf(0.044715f * z, z, 1.0f);  // 2 u
    return mul_limit(z, logistic(w));
  }
  if constexpr (ACT == ACT_SILU) return mul_limit(z, logistic(z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);  // (keeps NaN)
  if constexpr (ACT == ACT_GELU) {
    float e;
    const float q = normal_tail(z, &e);
    return (z < 0.0f ? q : 1.0f - q) + mul_limit(z, 0.39894228040143268f * e);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    const float zz = z * z;
    const float s = logistic(1.59576912160573071f * z * fmaf(0.044715f, zz, 1.0f));
    const float r = s * (1.0f - s);  // 0 wherever z * z overflows
    return s + mul_limit(1.59576912160573071f * z * fmaf(0.134145f, zz, 1.0f), r);
  }
  if constexpr (ACT == ACT_SILU) {
    const float s = logistic(z);
    return s + mul_limit(z, s * (1.0f - s));
  }
  return 1.0f;
}

// The 16-bit value in the low or high half of a word, in FP32.
template <typename T>
__device__ __forceinline__ float unpack(uint32_t w, int half);
template <>
__device__ __forceinline__ float unpack<_Float16>(uint32_t w, int half) {
  return (float)__builtin_bit_cast(f16x2, w)[half];
}
template <>
__device__ __forceinline__ float unpack<__bf16>(uint32_t w, int half) {
  return __builtin_bit_cast(float, half ? w & 0xffff0000u : w << 16);
}

// W words (2 W consecutive 16-bit values) of a row at column col of `cols`;
// columns at or past it read zeros.  One access of 4 W bytes wherever they
// are all inside, at any alignment: rows of odd lengths take no more
// instructions than aligned ones (element by element, a 777 x 1001 gradient
// call took 51 us).
template <int W>
__device__ __forceinline__ void load_row(const uint16_t* row, int col, int cols,
                                         uint32_t (&w)[W]) {
  const uint16_t* p = row + col;
  if (col + 2 * W <= cols) {
    if constexpr (W == 4) {
      const u32x4 v = *(const u32x4_any*)p;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = v[k];
    } else {
      const u32x2 v = *(const u32x2_any*)p;
      w[0] = v[0];
      w[1] = v[1];
    }
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t lo = col + 2 * k < cols ? p[2 * k] : 0u;
      const uint32_t hi = col + 2 * k + 1 < cols ? p[2 * k + 1] : 0u;
      w[k] = lo | (hi << 16);
    }
  }
}

template <int W>
__device__ __forceinline__ void store_row(uint16_t* row, int col, int cols,
                                          const uint32_t (&w)[W]) {
  uint16_t* p = row + col;
  if (col + 2 * W <= cols) {
    if constexpr (W == 4)
      __builtin_nontemporal_store((u32x4){w[0], w[1], w[2], w[3]}, (u32x4_any*)p);
    else
      __builtin_nontemporal_store((u32x2){w[0], w[1]}, (u32x2_any*)p);
  } else {
#pragma unroll
    for (int k = 0; k < 2 * W; ++k)
      if (col + k < cols) p[k] = (uint16_t)(w[k >> 1] >> ((k & 1) * 16));
  }
}

// v = f(v) over an R x C block of values, or v *= f(z) (F: act_slope).  The
// switch on the activation stands outside the loops: one uniform branch for
// the block.
template <int ACT, int R, int C>
__device__ __forceinline__ void act_block(float (&v)[R][C]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) v[r][c] = act_value<ACT>(v[r][c]);
}
template <typename T, int ACT, int R, int C>
__device__ __forceinline__ void slope_block(float (&v)[R][C], const uint32_t (&z)[R][C / 2]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) v[r][c] *= act_slope<ACT>(unpack<T>(z[r][c >> 1], c & 1));
}
template <int R, int C>
__device__ __forceinline__ void apply_act(int act, float (&v)[R][C]) {
  switch (act) {
    case ACT_RELU: act_block<ACT_RELU>(v); break;
    case ACT_GELU: act_block<ACT_GELU>(v); break;
    case ACT_GELU_TANH: act_block<ACT_GELU_TANH>(v); break;
    case ACT_SILU: act_block<ACT_SILU>(v); break;
    default: break;
  }
}
template <typename T, int R, int C>
__device__ __forceinline__ void apply_slope(int act, float (&v)[R][C], const uint32_t (&z)[R][C / 2]) {
  switch (act) {
    case ACT_RELU: slope_block<T, ACT_RELU>(v, z); break;
    case ACT_GELU: slope_block<T, ACT_GELU>(v, z); break;
    case ACT_GELU_TANH: slope_block<T, ACT_GELU_TANH>(v, z); break;
    case ACT_SILU: slope_block<T, ACT_SILU>(v, z); break;
    default: break;
  }
}

}  // namespace dg
