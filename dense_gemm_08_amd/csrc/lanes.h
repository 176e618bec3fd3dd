// lanes.h -- reductions over a wave's lanes (device side): maxima, minima and
// sums over 16 neighbouring lanes, or all 64, that every one of them receives.
// Within 16 lanes by DPP moves (an ALU operand read from another lane, no trip
// through LDS): lanes that differ in bit 0, then in bit 1, then the mirrored
// half row and row, whose quads already agree.  The order of a sum is fixed, and
// all lanes form the same bits.  All lanes of the wave must be active.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace dg {

// x of another lane of the row (all these patterns read lanes that there are).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ int dpp_move(int x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xf, 0xf, true);
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

// x of the even rows of 16 (S 16) or of the first two (S 32), `which` 0, or of the
// others, 1, in both rows of a pair: v_permlane16_swap and v_permlane32_swap of x
// with itself.
template <int S>
__device__ __forceinline__ uint32_t across(uint32_t x, int which) {
  typedef uint32_t pair __attribute__((ext_vector_type(2)));
  if constexpr (S == 16)
    return __builtin_bit_cast(pair, __builtin_amdgcn_permlane16_swap(x, x, false, false))[which];
  else
    return __builtin_bit_cast(pair, __builtin_amdgcn_permlane32_swap(x, x, false, false))[which];
}
template <int S>
__device__ __forceinline__ int across(int x, int which) {
  return (int)across<S>((uint32_t)x, which);
}
template <int S>
__device__ __forceinline__ float across(float x, int which) {
  return __builtin_bit_cast(float, across<S>(__builtin_bit_cast(uint32_t, x), which));
}
template <int S>
__device__ __forceinline__ double across(double x, int which) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = across<S>((uint32_t)b, which), hi = across<S>((uint32_t)(b >> 32), which);
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
    x = op(across<16>(x, 0), across<16>(x, 1));
    x = op(across<32>(x, 0), across<32>(x, 1));
  }
  return x;
}

// (whole numbers: max and min take a DPP operand)
template <typename X>
__device__ __forceinline__ X larger(X a, X b) {
  if constexpr (std::is_integral_v<X>)
    return max(a, b);
  else
    return b > a ? b : a;
}
template <int L, typename X>
__device__ __forceinline__ X max_lanes(X x) {
  return reduce_lanes<L>(x, [](X a, X b) { return larger(a, b); });
}
template <int L>
__device__ __forceinline__ int min_lanes(int x) {
  return reduce_lanes<L>(x, [](int a, int b) { return min(a, b); });
}
template <int L, typename X>
__device__ __forceinline__ X sum_lanes(X x) {
  return reduce_lanes<L>(x, [](X a, X b) { return a + b; });
}

// The sum of x over the lanes up to this one in its row of 16, and in the wave.
__device__ __forceinline__ int sum_up_to_row(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);  // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  return x;
}
__device__ __forceinline__ int sum_up_to(int x) {
  x = sum_up_to_row(x);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast 15, into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast 31, into rows 2 and 3
  return x;
}
// x of the next lane of the row; 0 in its last.
__device__ __forceinline__ uint32_t from_next(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x101, 0xf, 0xf, true);  // row_shl 1
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_move(uint64_t x) {
  return dpp_move<CTRL>((uint32_t)x) | ((uint64_t)dpp_move<CTRL>((uint32_t)(x >> 32)) << 32);
}

template <int S>
__device__ __forceinline__ uint64_t across(uint64_t x, int which) {
  return across<S>((uint32_t)x, which) | ((uint64_t)across<S>((uint32_t)(x >> 32), which) << 32);
}

// x of the lane whose number differs in bit D alone (D 16 and 32: of the wave).
template <int D, typename X>
__device__ __forceinline__ X other(X x) {
  if constexpr (D == 1) return dpp_move<0xB1>(x);
  if constexpr (D == 2) return dpp_move<0x4E>(x);
  if constexpr (D == 4) return dpp_move<0x1B>(dpp_move<0x141>(x));  // mirrored by 8, then by 4
  if constexpr (D == 8) return dpp_move<0x128>(x);                  // row_ror 8
  const bool high = ((int)threadIdx.x & D) != 0;
  const X a = across<D>(x, 0), b = across<D>(x, 1);
  return high ? a : b;
}
// x of the lane mirrored within blocks of N lanes.
template <int N, typename X>
__device__ __forceinline__ X mirrored(X x) {
  if constexpr (N == 2) return dpp_move<0xB1>(x);
  if constexpr (N == 4) return dpp_move<0x1B>(x);
  if constexpr (N == 8) return dpp_move<0x141>(x);
  if constexpr (N == 16) return dpp_move<0x140>(x);
  if constexpr (N == 32) return other<16>(dpp_move<0x140>(x));
  if constexpr (N == 64) return other<32>(other<16>(dpp_move<0x140>(x)));
}

// A step of a bitonic network that sorts in descending order: of a lane and its
// partner (which holds y), the lower one, whose bit BIT is clear, keeps the
// larger value.
template <int BIT, typename X>
__device__ __forceinline__ X sort_step(X x, X y) {
  const bool upper = ((int)threadIdx.x & BIT) != 0;
  if constexpr (sizeof(X) == 4) {
    return upper ? min(x, y) : max(x, y);
  } else {
    return (y > x) != upper ? y : x;
  }
}
// A bitonic run of 2 D lanes in descending order.
template <int D, typename X>
__device__ __forceinline__ X sort_bitonic(X x) {
  x = sort_step<D>(x, other<D>(x));
  if constexpr (D > 1) x = sort_bitonic<D / 2>(x);
  return x;
}
// The values of N neighbouring lanes in descending order.
template <int N, typename X>
__device__ __forceinline__ X sorted_lanes(X x) {
  if constexpr (N > 2) x = sorted_lanes<N / 2>(x);
  x = sort_step<N / 2>(x, mirrored<N>(x));
  if constexpr (N > 2) x = sort_bitonic<N / 4>(x);
  return x;
}
// The 16 largest of two rows that are in order, in order.
template <typename X>
__device__ __forceinline__ X merged_in_row(X x, X y) {
  const X z = mirrored<16>(y);
  return sort_bitonic<8>(z > x ? z : x);
}

// Values that lanes of this wave left in LDS for each other: the accesses after
// this follow those before it (a wave's LDS accesses complete in order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace dg
