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

// The activations and their slopes on a block of C values, as a sequence of
// stages over the whole block that the fences keep apart: done value by value,
// every exponential and reciprocal is waited for at once (4096 x 4096 x 512
// with SILU 29 us value by value, 25 in stages, 23 without an activation).
// Infinite z: the factor that tends to 0
// is 0 exactly there (and wherever |z| > FAR), so z is replaced by a finite
// value in the product with it; NaN comes through that factor.
constexpr float FAR = 1e4f;
__device__ __forceinline__ float not_far_below(float z) {
  return __builtin_amdgcn_fmed3f(z, -FAR, __builtin_inff());
}

template <int C>
__device__ __forceinline__ void stage_logistic(float (&w)[C]) {
  fence();
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] = __builtin_amdgcn_exp2f(w[c]);
  fence();
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] += 1.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] = __builtin_amdgcn_rcpf(w[c]);
  fence();
}

// w = s(a z) for SILU (a z = z) or s(2 u) for GELU_TANH; exp2's argument is
// -log2(e) times that.
template <int ACT, int C>
__device__ __forceinline__ void block_logistic(const float (&z)[C], float (&w)[C]) {
  constexpr float L2E = 1.44269504088896341f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (ACT == ACT_SILU)
      w[c] = z[c] * -L2E;
    else  // 2 u = z (1.5957.. + 0.0713.. z^2), 1.5957.. = 2 sqrt(2 / pi)
      w[c] = z[c] * fmaf(z[c] * z[c], -L2E * 0.07135481283f, -L2E * 1.59576912161f);
  }
  stage_logistic(w);
}

// The normal distribution: with y = |z| / sqrt(2), F(-|z|) = exp(-y^2) q(y),
// q(y) = erfc(y) exp(y^2) / 2.  q is a polynomial in t = 1 / (1 + 0.375 y),
// fitted here for least relative error over 0 <= y <= 14 (1.4e-6, so the
// negative tail keeps its relative precision down to the smallest 16-bit
// results, where 1 + erf(z / sqrt(2)) would cancel).  Gives F(-|z|) and
// exp(-z^2 / 2).
template <int C>
__device__ __forceinline__ void block_normal(const float (&z)[C], float (&tail)[C],
                                             float (&gauss)[C]) {
  float t[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    t[c] = fmaf(0.26516504294495533f, fabsf(z[c]), 1.0f);  // 0.375 / sqrt(2)
    gauss[c] = z[c] * z[c] * -0.72134752044448170f;        // -log2(e) / 2
  }
  fence();
#pragma unroll
  for (int c = 0; c < C; ++c) t[c] = __builtin_amdgcn_rcpf(t[c]);
#pragma unroll
  for (int c = 0; c < C; ++c) gauss[c] = __builtin_amdgcn_exp2f(gauss[c]);
  fence();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float q = 0.5f * -0.13092039f;
    q = fmaf(q, t[c], 0.5f * 0.37347726f);
    q = fmaf(q, t[c], 0.5f * -0.10964101f);
    q = fmaf(q, t[c], 0.5f * 0.26908684f);
    q = fmaf(q, t[c], 0.5f * 0.17187412f);
    q = fmaf(q, t[c], 0.5f * 0.21471366f);
    q = fmaf(q, t[c], 0.5f * 0.21141088f);
    tail[c] = gauss[c] * (t[c] * q);
  }
}

// z = act(z)
template <int ACT, int C>
__device__ __forceinline__ void block_value(float (&z)[C]) {
  if constexpr (ACT == ACT_RELU) {
#pragma unroll
    for (int c = 0; c < C; ++c) z[c] = z[c] < 0.0f ? 0.0f : z[c];  // (keeps NaN)
  } else if constexpr (ACT == ACT_GELU) {
    float q[C], e[C];
    block_normal(z, q, e);
#pragma unroll
    for (int c = 0; c < C; ++c) z[c] = not_far_below(z[c]) * (z[c] < 0.0f ? q[c] : 1.0f - q[c]);
  } else {
    float s[C];
    block_logistic<ACT>(z, s);
#pragma unroll
    for (int c = 0; c < C; ++c) z[c] = not_far_below(z[c]) * s[c];
  }
}

// d = act'(z)
template <int ACT, int C>
__device__ __forceinline__ void block_slope(const float (&z)[C], float (&d)[C]) {
  if constexpr (ACT == ACT_RELU) {
#pragma unroll
    for (int c = 0; c < C; ++c) d[c] = z[c] > 0.0f ? 1.0f : (z[c] <= 0.0f ? 0.0f : z[c]);
  } else if constexpr (ACT == ACT_GELU) {
    float q[C], e[C];
    block_normal(z, q, e);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float near = __builtin_amdgcn_fmed3f(z[c], -FAR, FAR);
      d[c] = fmaf(0.39894228040143268f * near, e[c], z[c] < 0.0f ? q[c] : 1.0f - q[c]);
    }
  } else {
    float s[C];
    block_logistic<ACT>(z, s);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float near = __builtin_amdgcn_fmed3f(z[c], -FAR, FAR);
      // d(2 u)/dz = 1.5957.. + 3 * 0.0713.. z^2
      if constexpr (ACT == ACT_GELU_TANH)
        near *= fmaf(near * near, 3.0f * 0.07135481283f, 1.59576912161f);
      d[c] = fmaf(near, fmaf(-s[c], s[c], s[c]), s[c]);
    }
  }
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

// v = act(v) over R rows of C values, or v *= act'(z).  The switch on the
// activation stands outside the loops: one uniform branch for the block.
// Two rows at a time: enough values to cover the latencies, few enough for the
// registers beside a 256 x 256 tile's accumulators.
template <int ACT, int R, int C>
__device__ __forceinline__ void act_block(float (&v)[R][C]) {
  constexpr int H = R > 1 ? 2 : 1;
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += H) {
    float x[H * C];
#pragma unroll
    for (int k = 0; k < H * C; ++k) x[k] = v[r0 + k / C][k % C];
    block_value<ACT>(x);
#pragma unroll
    for (int k = 0; k < H * C; ++k) v[r0 + k / C][k % C] = x[k];
    fence();
  }
}
template <typename T, int ACT, int R, int C>
__device__ __forceinline__ void slope_block(float (&v)[R][C], const uint32_t (&z)[R][C / 2]) {
  constexpr int H = R > 1 ? 2 : 1;
#pragma unroll
  for (int r0 = 0; r0 < R; r0 += H) {
    float x[H * C], d[H * C];
#pragma unroll
    for (int k = 0; k < H * C; ++k) x[k] = unpack<T>(z[r0 + k / C][k % C >> 1], k & 1);
    block_slope<ACT>(x, d);
#pragma unroll
    for (int k = 0; k < H * C; ++k) v[r0 + k / C][k % C] *= d[k];
    fence();
  }
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

// The forward epilogue of C scaled sums of a row, from column col on: bias, Z,
// activation, residual.
template <typename O, int C>
__device__ __forceinline__ void finish_row(const Epilogue& e, int group, int64_t row, int col, int N,
                                           float (&x)[1][C]) {
  uint32_t w[C / 2];
  if (e.bias != nullptr) {
    load_row<C / 2>(e.bias + group * e.bias_stride, col, N, w);
#pragma unroll
    for (int k = 0; k < C; ++k) x[0][k] += unpack<O>(w[k >> 1], k & 1);
  }
  if (e.z != nullptr) {
#pragma unroll
    for (int k = 0; k < C / 2; ++k) w[k] = pack2<O>(x[0][2 * k], x[0][2 * k + 1]);
    store_row<C / 2>(e.z + row * e.ldz, col, N, w);
  }
  apply_act(e.act, x);
  if (e.res != nullptr) {
    load_row<C / 2>(e.res + row * e.ldr, col, N, w);
#pragma unroll
    for (int k = 0; k < C; ++k) x[0][k] += unpack<O>(w[k >> 1], k & 1);
  }
}

}  // namespace dg
