// lanes.h -- reductions over a wave's lanes (device side): maxima, minima and
// sums over 16 neighbouring lanes, or all 64, that every one of them receives.
// Within 16 lanes by DPP moves (an ALU operand read from another lane, no trip
// through LDS): lanes that differ in bit 0, then in bit 1, then the mirrored
// half row and row, whose quads already agree.  The order of a sum is fixed, and
// all lanes form the same bits.  All lanes of the wave must be active.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ int dpp_move(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
  return __builtin_bit_cast(float, dpp_move<CTRL>(__builtin_bit_cast(uint32_t, x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = dpp_move<CTRL>((uint32_t)b), hi = dpp_move<CTRL>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, lo | (hi << 32));
}

// x of L lanes (16 or 64) combined by op(a, b), a commutative one.
template <int L, typename X, typename Op>
__device__ __forceinline__ X reduce_lanes(X x, Op&& op) {
  static_assert(L == 16 || L == 64, "rows of 16 lanes, or the wave");
  x = op(x, dpp_move<0xB1>(x));   // quad_perm 1 0 3 2
  x = op(x, dpp_move<0x4E>(x));   // quad_perm 2 3 0 1
  x = op(x, dpp_move<0x141>(x));  // row_half_mirror
  x = op(x, dpp_move<0x140>(x));  // row_mirror
  if constexpr (L == 64) {
    x = op(x, (X)__shfl_xor(x, 16));
    x = op(x, (X)__shfl_xor(x, 32));
  }
  return x;
}

template <int L, typename X>
__device__ __forceinline__ X max_lanes(X x) {
  return reduce_lanes<L>(x, [](X a, X b) { return b > a ? b : a; });
}
template <int L, typename X>
__device__ __forceinline__ X min_lanes(X x) {
  return reduce_lanes<L>(x, [](X a, X b) { return b < a ? b : a; });
}
template <int L, typename X>
__device__ __forceinline__ X sum_lanes(X x) {
  return reduce_lanes<L>(x, [](X a, X b) { return a + b; });
}

}  // namespace dg
