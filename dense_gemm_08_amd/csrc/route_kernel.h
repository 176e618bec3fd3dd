// route_kernel.h -- routing of tokens to experts on the MI355X (gfx950): the
// choice of every token's experts from its logits, their weights, and the
// dispatch (the order of the chosen rows by expert), with the weights'
// gradient.
//
// A token is handled by L neighbouring lanes (16, or a wave beyond 512 experts),
// PER logits a lane in registers.  The
// dispatch is a counting sort: a workgroup takes 64 tokens at a time and marks
// in a 64-bit word per expert which of them chose it (LDS atomics of an OR,
// whose order changes nothing), so that a choice's rank among them is a count of
// the bits below its token's.  The order of the rows, by expert and then by
// token, is thus fixed.
//
// Scores are compared in 32 bits where these decide.  With a bias (or sums of
// scores for groups) two candidates may lie closer together than the rounding
// errors of their scores; such a token's choice is made again in 64 bits, by a
// wave, so that it does not depend on how a 32-bit exponential rounds.  Without
// them the logits themselves are compared, which is exact.
//
// Bound by instructions and their latencies, not by memory: 16384 tokens of 256
// FP32 logits (17 MB, 3 us), 8 chosen, take 9 us ranked by their logits, 14.5 with
// a logistic and a bias, 18.6 with 4 of 8 groups: 5 to read and to mark what is
// broken, 2.6 the scores, 3.2 the groups, 2 the choice, 1 the weights; VALU busy
// 0.67 of that.  3 to 5 us of the last two are the tokens whose choice 32 bits do
// not settle (each 5 us of its wave), whose waves end last: one in 3000 with random
// logits and biases.  Equal candidates count among them, and where logits of few
// bits meet a bias of zeros these are many: 37% of the tokens in BF16, 5% in FP16,
// whose whole call then takes 38 us (47 with the groups) and 28 (34) against 19
// (24) with FP32 logits or random biases; with biases in steps of 0.05 7% in BF16,
// 27 us (32).  (One expert after the other found by a maximum over all, with the
// 64-bit form in line: 79.)
// route_place then takes 5.6 us.
// 1024 experts, found one after the other by a wave a token, take 50 us ranked, 67
// with a logistic and a bias, 86 with 4 of 8 groups (67 MB, 13 us); with BF16 logits,
// whose equal ones are looked up again, 80, 94 and 109.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cdna_ops.h"
#include "epilogue.h"
#include "lanes.h"
#include "plan_experts.h"

namespace dg {

struct RouteParams {
  const void* logits;
  const float* bias;   // or null
  float* weights;      // T x k
  int32_t* experts;    // T x k
  int32_t* places;     // T x k
  int32_t* ends;       // E
  int32_t* tokens;     // T k
  uint32_t* counts;    // choices per block and expert, two in a word (null: one block)
  int64_t ld;
  int T, E, k;
  int sigmoid, renorm;
  float scale;
  int ranked;          // no bias: the logits rank the experts
  int groups, group_size, top_groups, group_top;
  int group_lanes[2];  // lanes of 16, of 64, that look for a group's best: powers of two
  int group_inverse;   // ceil(2^20 / group_size): e * that >> 20 is e's group
  int k_inverse;       // ceil(2^20 / k): i * that >> 20 is i / k for i < 64 k
  int chunks;          // chunks of 64 tokens per block
};

// One token's logits in FP32, spread over L lanes: l[i] is expert i L + lane's;
// -inf past E (and everywhere for a token that there is not).
template <typename F, int L, int PER>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&l)[PER]) {
  const F* row = (const F*)p.logits + (t < p.T ? t : 0) * p.ld;
  if (p.E == L * PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = (float)row[i * L + lane];
  } else {
    // (the last expert's where there is none: no branch per logit)
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = (float)row[min(i * L + lane, p.E - 1)];
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = i * L + lane < p.E ? l[i] : -__builtin_inff();
  }
  if (t >= p.T) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = -__builtin_inff();
  }
}

// Whether one of a token's logits is NaN or +inf.
template <int L, int PER>
__device__ __forceinline__ bool broken_row(const float (&l)[PER]) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) bad |= !(l[i] < __builtin_inff());
  return max_lanes<L>(bad ? 1 : 0) != 0;
}
// The largest of a token's logits, 0 if there is none; of use for a softmax.
template <int L, int PER>
__device__ __forceinline__ float top_logit(const RouteParams& p, const float (&l)[PER]) {
  if (p.sigmoid) return 0.0f;
  float m = l[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = l[i] > m ? l[i] : m;
  m = max_lanes<L>(m);
  return m > -__builtin_inff() ? m : 0.0f;
}

// The scores of a token's experts plus their bias, -inf where one cannot be
// chosen; with the logits themselves where these decide (RouteParams::ranked).
// Returns by how much two of them have to differ, next to 2^-23 of their size,
// for their order to be sure (sums of two: by twice as much, next to 2^-21): in
// 32 bits a logistic's error is below 2^-22 (its exponential's, at most 2^-24, the
// reciprocal's 2^-23, the sum's 2^-24), a softmax's 2^-18 of the largest (its
// sum's, above all), the bias's sum rounds by 2^-24 of it, and a difference has
// two of each.
template <typename X, int L, int PER>
__device__ __forceinline__ X choice_scores(const RouteParams& p, const float (&l)[PER], int lane,
                                           float top, X (&c)[PER]) {
  const X NONE = -(X)__builtin_inff();
  if (p.ranked && p.group_top == 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i];
    return 0;
  }
  constexpr bool FAST = sizeof(X) == 4;
  constexpr float L2E = 1.44269504088896341f;
  X near = (X)0x1p-21;
  if (!p.sigmoid) {
    X sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (FAST)
        c[i] = __builtin_amdgcn_exp2f((l[i] - top) * L2E);
      else
        c[i] = exp((X)l[i] - (X)top);
      sum += c[i];
      if constexpr (!FAST && PER > 4) fence();  // (one after the other: they take many registers)
    }
    const X part = 1 / sum_lanes<L>(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] *= part;
    near = part * (X)0x1p-17;
  } else if constexpr (FAST) {
    float e[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) e[i] = __builtin_amdgcn_exp2f(l[i] * -L2E);
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = 1 / (1 + exp(-(X)l[i]));
      if constexpr (PER > 4) fence();
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * L + lane;
    if (p.bias != nullptr) c[i] += (X)p.bias[min(e, p.E - 1)];
    if (!(l[i] > -__builtin_inff()) || !(c[i] > NONE)) c[i] = NONE;
  }
  return near;
}

// 32-bit values as whole numbers in the same order (no NaN; both zeros alike),
// and back.
constexpr int KEY_NONE = (int)0x807fffff;  // -inf
__device__ __forceinline__ int key_of(float x) {
  const int b = __builtin_bit_cast(int, x + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int key) {
  return __builtin_bit_cast(float, key ^ ((key >> 31) & 0x7fffffff));
}
// A value and its index as one number: the larger of two stands for the larger
// value, of equal ones for the lower index.  0 is none (and -inf none).
__device__ __forceinline__ uint64_t ranked_pair(float x, int index) {
  const int key = key_of(x);
  return key > KEY_NONE ? ((uint64_t)((uint32_t)key ^ 0x80000000u) << 32) | ~(uint32_t)index : 0;
}
__device__ __forceinline__ float pair_value(uint64_t pair) {
  return pair != 0 ? value_of((int)((uint32_t)(pair >> 32) ^ 0x80000000u)) : -__builtin_inff();
}
__device__ __forceinline__ int pair_index(uint64_t pair) { return (int)~(uint32_t)pair; }

// The 16 bits of a wave's ballot that are this lane's row's.
__device__ __forceinline__ uint32_t row_bits(uint64_t ballot) {
  const int lane = (int)threadIdx.x & 63;
  const uint32_t half = lane < 32 ? (uint32_t)ballot : (uint32_t)(ballot >> 32);
  return lane & 16 ? half >> 16 : half & 0xffffu;
}
// x of lane n (the same in all lanes) of this lane's row, or of the wave.
template <int L>
__device__ __forceinline__ int at_lane(int x, int n) {
  if constexpr (L == 64) return __builtin_amdgcn_readlane(x, n);
  return __builtin_amdgcn_ds_bpermute((((int)threadIdx.x & 48) | n) << 2, x);
}
template <int L>
__device__ __forceinline__ uint64_t at_lane(uint64_t x, int n) {
  return (uint32_t)at_lane<L>((int)(uint32_t)x, n) |
         ((uint64_t)(uint32_t)at_lane<L>((int)(uint32_t)(x >> 32), n) << 32);
}

// The largest x of L lanes.  In 32 bits as whole numbers, whose maximum takes one
// instruction with the other lane's as its operand (16384 tokens of 1024 experts
// with a bias 57.8 us, 56.0 so).  In 64 bits as it stands: by x rounded to FP32
// first, and in full where lanes are equal so, a token took 5.6 us for 5.
template <int L, typename X>
__device__ __forceinline__ X largest(X x) {
  if constexpr (sizeof(X) == 4)
    return value_of(max_lanes<L>(key_of(x)));
  else
    return max_lanes<L>(x);
}

// The larger of two numbers (32 bits: in one instruction, by the median with
// infinity), and the two largest of three.
__device__ __forceinline__ float larger_of(float a, float b) {
  return __builtin_amdgcn_fmed3f(a, b, __builtin_inff());
}
__device__ __forceinline__ void take_top(float x, float& first, float& second) {
  second = __builtin_amdgcn_fmed3f(x, first, second);
  first = larger_of(first, x);
}
__device__ __forceinline__ void take_top(double x, double& first, double& second) {
  second = fmax(second, fmin(first, x));
  first = fmax(first, x);
}

// Whether a, the larger, is not surely larger than b; size: that of what they
// were summed from.
template <typename X>
__device__ __forceinline__ bool too_close(X a, X b, X near, X size) {
  if (sizeof(X) == 8 || !(b > -(X)__builtin_inff())) return false;
  return !(a - b > near + (X)0x1p-23 * size);  // (so is a difference that is no number)
}

// Where expert e's value lies in LDS: a gap every 16, so that groups whose sizes
// are powers of two do not begin in the same few banks (256 experts in 8 groups:
// 5 of 6 LDS cycles were conflicts).
__device__ __forceinline__ constexpr int lds_at(int e) { return e + (e >> 4); }

// Takes the experts outside the best groups from c.  `lds`: E values of this
// token's, which receive c as it was.  Returns whether rounding could change
// that.
template <typename X, int L, int PER>
__device__ __forceinline__ bool limit_groups(const RouteParams& p, int lane, X near, X* lds, X (&c)[PER]) {
  const X NONE = -(X)__builtin_inff();
#pragma unroll
  for (int i = 0; i < PER; ++i) lds[lds_at(i * L + lane)] = c[i];
  wave_lds_order();
  // A group's two best, found by `share` neighbouring lanes (up to 16, a power
  // of two) where there are no more groups than lanes; else several groups a
  // lane.
  constexpr int GS = (ROUTE_MOST_GROUPS + L - 1) / L;
  X value[GS], size = 0;
  const int share = p.group_lanes[L == 64];
#pragma unroll
  for (int n = 0; n < GS; ++n) {
    const int g = n * L + lane / share;
    X first = NONE, second = NONE;
    if (g < p.groups) {
      const int end = (g + 1) * p.group_size;
#pragma unroll 8
      for (int e = g * p.group_size + (lane & (share - 1)); e < end; e += share)
        take_top(lds[lds_at(e)], first, second);
    }
    auto join = [&](X f, X s) {
      take_top(f, first, second);
      second = fmax(second, s);
    };
    if (share > 1) join(dpp_move<0xB1>(first), dpp_move<0xB1>(second));
    if (share > 2) join(dpp_move<0x4E>(first), dpp_move<0x4E>(second));
    if (share > 4) join(dpp_move<0x141>(first), dpp_move<0x141>(second));
    if (share > 8) join(dpp_move<0x140>(first), dpp_move<0x140>(second));
    const bool two = p.group_top > 1 && second > NONE;
    value[n] = two ? first + second : first;
    // (a sum below FP32's range is still a group's that can be chosen)
    if (sizeof(X) == 4 && two) value[n] = fmax(value[n], -(X)3.402823466e38f);
    if (first > NONE) size = fmax(size, fmax(fabs(first), two ? fabs(second) : (X)0));
    if (share > 1) break;
  }
  const bool exact = sizeof(X) == 8 || (p.ranked && p.group_top == 1);
  bool unsure = false;
  if constexpr (sizeof(X) == 4) {
    if (p.groups <= L) {
      // the groups put in order all at once, each by the first of its lanes
      const uint64_t own = (lane & (share - 1)) == 0 ? ranked_pair(value[0], lane) : 0;
      const uint64_t order = sorted_lanes<L>(own);
      // (top_groups < groups <= L)
      const uint64_t last = at_lane<L>(order, p.top_groups - 1), next = at_lane<L>(order, p.top_groups);
      const uint64_t in = __ballot(own != 0 && own >= last);
      const uint64_t stays = L == 64 ? in : row_bits(in);  // bit (group * share)
      // (the size of the two in question: others may be masked by huge biases)
      if (!exact) {
        size = max_lanes<L>(own == last || own == next ? size : (X)0);
        unsure = too_close(pair_value(last), pair_value(next), 2 * near, 4 * size);
      }
      auto keep = [&](int i, int g) {
        const int stay = L == 16 ? (int)((uint32_t)stays << (31 - g * share)) >> 31  // all bits, or none
                                 : -(int)(stays >> (g * share) & 1);
        c[i] = __builtin_bit_cast(float, (__builtin_bit_cast(int, c[i]) & stay) |
                                             (__builtin_bit_cast(int, (float)NONE) & ~stay));
      };
      if (p.group_size % L == 0) {  // (an element's group is the same one in all lanes)
#pragma unroll
        for (int i = 0; i < PER; ++i) keep(i, min(i * L * p.group_inverse >> 20, p.groups - 1));
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) keep(i, min((i * L + lane) * p.group_inverse >> 20, p.groups - 1));
      }
      return unsure;
    }
  }
  if (!exact) size = max_lanes<L>(size);
  uint64_t stays = 0;
  X least = 0;
  for (int n = 0; n <= p.top_groups; ++n) {
    X m = value[0];
    int at = lane / share;
#pragma unroll
    for (int i = 1; i < GS; ++i)
      if (share == 1 && value[i] > m) {
        m = value[i];
        at = i * L + lane;
      }
    const X best = largest<L>(m);
    if (!(best > NONE)) break;
    if (n == p.top_groups) {
      unsure = !exact && too_close(least, best, 2 * near, 4 * size);
      break;
    }
    least = best;
    const int g = min_lanes<L>(m == best ? at : 1 << 30);
    stays |= 1ull << (g & 63);
#pragma unroll
    for (int i = 0; i < GS; ++i)
      if ((share > 1 ? lane / share : i * L + lane) == g) value[i] = NONE;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = (i * L + lane) * p.group_inverse >> 20 & 63;
    if (!(stays >> g & 1)) c[i] = NONE;
  }
  return unsure;
}

// The k best of c, found one after the other; sel receives their experts (-1
// where there is none).  Returns whether rounding could change the choice or its
// order.
template <typename X, int L, int PER>
__device__ __forceinline__ bool pick_in_turn(const RouteParams& p, int lane, X near, X (&c)[PER], int* sel) {
  const X NONE = -(X)__builtin_inff();
  bool unsure = false;
  X before = 0;
  // (one more than there are choices, whose distance from the last counts)
  for (int j = 0; j <= p.k; ++j) {
    X m = c[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (c[i] > m) {
        m = c[i];
        at = i;
      }
    const X best = largest<L>(m);
    if (!p.ranked && j > 0) unsure |= too_close(before, best, near, (X)fmax(fabs(before), fabs(best)));
    before = best;
    if (j == p.k) break;
    int e;
    const uint64_t who = __ballot(m == best);
    if (L == 64 && __popcll(who) == 1) {  // (one lane has it)
      const int w = __builtin_ctzll(who);
      e = __builtin_amdgcn_readlane(at, w) * 64 + w;
    } else {
      e = min_lanes<L>(m == best ? at * L + lane : 1 << 30);
    }
    if (lane == 0) sel[j] = best > NONE ? e : -1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * L + lane == e) c[i] = NONE;
  }
  wave_lds_order();
  return unsure;
}

// The same in 32 bits for up to 15 of a row of 16 lanes, all at once: none of
// the k + 1 best is below the (k + 1)-th largest of the lanes' maxima, and few
// others are not (256 experts, 8 chosen: 14 expected).  These candidates' indices
// are gathered in LDS and put in order, two a lane at most, by a bitonic network.
// `lds`: the values c of this token, by expert.  *done is false, for the whole
// wave, if some token has more than 32.
template <int PER>
__device__ __forceinline__ bool pick_at_once(const RouteParams& p, int lane, float near, const float (&c)[PER],
                                             const float* lds, int* sel, bool* done) {
  static_assert(ROUTE_MOST_K >= 32, "sel holds the candidates first");
  float m = c[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) m = larger_of(m, c[i]);
  const float limit = value_of(max(at_lane<16>(sorted_lanes<16>(key_of(m)), p.k), KEY_NONE + 1));
  uint32_t bits = 0;
#pragma unroll
  for (int i = PER - 1; i >= 0; --i) bits = bits + bits + (c[i] >= limit ? 1 : 0);
  const int count = __popc(bits), total = sum_lanes<16>(count);
  int at = sum_up_to_row(count) - count;
  *done = __ballot(total > 32) == 0;
  if (!*done) return false;
  while (__ballot(bits != 0) != 0) {
    if (bits != 0) {
      sel[at++] = __builtin_ctz(bits) * 16 + lane;
      bits &= bits - 1;
    }
  }
  wave_lds_order();
  uint64_t best = 0;
  if (lane < total) {
    const int e = sel[lane];
    best = ranked_pair(lds[lds_at(e)], e);
  }
  best = sorted_lanes<16>(best);
  if (__ballot(total > 16) != 0) {
    uint64_t more = 0;
    if (lane + 16 < total) {
      const int e = sel[lane + 16];
      more = ranked_pair(lds[lds_at(e)], e);
    }
    best = merged_in_row(best, sorted_lanes<16>(more));
  }
  wave_lds_order();
  if (lane < p.k) sel[lane] = best != 0 ? pair_index(best) : -1;
  wave_lds_order();
  if (p.ranked) return false;
  const uint64_t next = from_next((uint32_t)best) | ((uint64_t)from_next((uint32_t)(best >> 32)) << 32);
  const float v = pair_value(best), w = pair_value(next);
  return max_lanes<16>(lane < p.k && too_close(v, w, near, fmaxf(fabsf(v), fabsf(w))) ? 1 : 0) != 0;
}

// The scores that weights are made of.  With renorm a factor common to the
// chosen is left out, so that none underflows beside larger ones: a softmax's
// exp(-b.top), a logistic's where all chosen logits are negative.
struct ScoreBase {
  float top;
  float sum;  // the softmax's sum over all experts, or 1
};
__device__ __forceinline__ float score_of(const RouteParams& p, float l, const ScoreBase& b) {
  if (!p.sigmoid) return expf(l - b.top) / b.sum;
  if (l > 0.0f) return 1.0f / (1.0f + expf(-l));
  return expf(l - b.top) / (1.0f + expf(l));
}
template <int L, int PER>
__device__ __forceinline__ ScoreBase score_base(const RouteParams& p, const float (&l)[PER], float top,
                                                float top_chosen) {
  ScoreBase b = {0.0f, 1.0f};
  if (p.renorm) {
    b.top = p.sigmoid ? fminf(top_chosen, 0.0f) : top_chosen;
  } else if (!p.sigmoid) {
    b.top = top;
    // (the hardware's exponential: an error of 2^-22 in a term that counts)
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) s += __builtin_amdgcn_exp2f((l[i] - top) * 1.44269504088896341f);
    b.sum = sum_lanes<L>(s);
  }
  return b;
}

// A token's weights and experts from its choice, counted in `counts`; slot j is
// lane j mod L's.
template <typename F, int L, int PER>
__device__ __forceinline__ void finish_token(const RouteParams& p, int64_t t, int lane, const float (&l)[PER],
                                             float top, bool broken, const int* sel, int32_t* counts) {
  constexpr int SLOTS = (ROUTE_MOST_K + L - 1) / L;
  const F* row = (const F*)p.logits + t * p.ld;
  int e[SLOTS];
  float s[SLOTS], m = -__builtin_inff(), total = 0.0f;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    e[i] = i * L + lane < p.k && !broken ? sel[i * L + lane] : -1;
    s[i] = e[i] >= 0 ? (float)row[e[i]] : -__builtin_inff();
    m = fmaxf(m, s[i]);
    if (p.k <= (i + 1) * L) break;
  }
  const ScoreBase b = score_base<L, PER>(p, l, top, max_lanes<L>(m));
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    s[i] = e[i] >= 0 ? score_of(p, s[i], b) : 0.0f;
    total += s[i];
    if (p.k <= (i + 1) * L) break;
  }
  total = sum_lanes<L>(total);
  if (!p.renorm || total == 0.0f) total = 1.0f;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int j = i * L + lane;
    if (j >= p.k) break;
    p.weights[t * p.k + j] = broken ? __builtin_nanf("") : s[i] / total * p.scale;
    p.experts[t * p.k + j] = e[i];
    if (e[i] >= 0) atomicAdd(&counts[e[i]], 1);
  }
}

// The experts of the choices of the 64 tokens from t0 on (as many as there are),
// a thread's in registers; -1 behind them.
constexpr int HELD = ROUTE_MOST_K * 64 / ROUTE_THREADS;
struct HeldExperts {
  int e[HELD];
};
__device__ __forceinline__ HeldExperts load_experts(const RouteParams& p, int t0) {
  HeldExperts h;
  const int n = min(64, p.T - t0) * p.k;
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    const int i = u * ROUTE_THREADS + (int)threadIdx.x;
    h.e[u] = i < n ? p.experts[(int64_t)t0 * p.k + i] : -1;
  }
  return h;
}

// The order of those tokens' chosen rows: each choice's place, and its token
// there.  base[e]: the place of the first of them that chose e, moved on past the
// last at the end if there are more; mask: E words of zeros, then left so.
__device__ __forceinline__ void place_chunk(const RouteParams& p, int t0, const HeldExperts& h, int32_t* base,
                                            uint64_t* mask, bool more) {
  const int n = min(64, p.T - t0) * p.k;
  int t[HELD];
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    const int i = u * ROUTE_THREADS + (int)threadIdx.x;
    t[u] = (int)((uint32_t)i * (uint32_t)p.k_inverse >> 20);
    if (h.e[u] >= 0) atomicOr((unsigned long long*)&mask[h.e[u]], 1ull << t[u]);
    if (n <= (u + 1) * ROUTE_THREADS) break;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    const int i = u * ROUTE_THREADS + (int)threadIdx.x;
    if (i >= n) break;
    int at = -1;
    if (h.e[u] >= 0) {
      at = base[h.e[u]] + __popcll(mask[h.e[u]] & ((1ull << t[u]) - 1));
      p.tokens[at] = t0 + t[u];
    }
    p.places[(int64_t)t0 * p.k + i] = at;
  }
  if (!more) return;
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) {
    base[e] += __popcll(mask[e]);
    mask[e] = 0;
  }
  __syncthreads();
}

// The sum of v over the block's threads up to this one; *total: over all.
// scratch: one value per wave.
__device__ __forceinline__ int32_t scan_threads(int32_t v, int32_t* scratch, int32_t* total) {
  constexpr int WAVES_RT = ROUTE_THREADS / 64;
  static_assert(ROUTE_MOST_EXPERTS <= ROUTE_THREADS, "a thread per expert");
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  v = sum_up_to(v);
  if ((threadIdx.x & 63) == 63) scratch[wave] = v;
  __syncthreads();
  *total = 0;
#pragma unroll
  for (int w = 0; w < WAVES_RT; ++w) {
    const int32_t x = scratch[w];
    *total += x;
    v += w < wave ? x : 0;
  }
  return v;
}

// The choice: a block takes `chunks` times 64 tokens.  A lone block also makes
// the dispatch; otherwise each leaves its choices per expert in counts, for
// route_place.
template <typename F, int L, int PER>
__global__ __launch_bounds__(ROUTE_THREADS) void route_choose(RouteParams p) {
  constexpr int TPW = 64 / L, WAVES_RT = ROUTE_THREADS / 64;
  constexpr int AT_ONCE = ROUTE_THREADS / L, MOST = L * PER, ROOM = lds_at(MOST);
  // a wave's scores, by token (in 64 bits one token's)
  __shared__ __attribute__((aligned(16))) float area[WAVES_RT][(TPW < 2 ? 2 : TPW) * ROOM];
  __shared__ int sel[AT_ONCE][ROUTE_MOST_K];  // the chosen, in order
  __shared__ uint64_t mask[MOST];
  __shared__ int32_t base[MOST], scratch[WAVES_RT];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) {
    base[e] = 0;
    mask[e] = 0;
  }
  __syncthreads();
  const int first = (int)blockIdx.x * p.chunks * 64, tokens = min(p.T - first, p.chunks * 64);
  for (int t0 = 0; t0 < tokens; t0 += AT_ONCE) {
    uint64_t again;
    {
      // (the lane is read anew for each pass: what derives from it, biases and
      // groups among it, would otherwise be kept in registers over the loop)
      const int tid = opaque_tid(), lane = tid & (L - 1), sub = (tid & 63) / L, slot = tid / L;
      const int64_t t = (int64_t)first + t0 + slot;
      float l[PER], c[PER];
      load_logits<F, L, PER>(p, t, lane, l);
      const bool broken = broken_row<L, PER>(l);
      const float top = top_logit<L, PER>(p, l);
      const float near = choice_scores<float, L, PER>(p, l, lane, top, c);
      bool unsure = false, done = false;
      if (p.top_groups < p.groups) {
        unsure = limit_groups<float, L, PER>(p, lane, near, area[wave] + sub * ROOM, c);
        if (p.ranked && p.group_top > 1) {
          // (sums of scores chose the groups; within them the logits rank)
#pragma unroll
          for (int i = 0; i < PER; ++i) c[i] = c[i] > -__builtin_inff() ? l[i] : c[i];
        }
      }
      // (a wave of 64 lanes a token finds them in turn: the network of its
      // candidates would spill registers, 1024 experts, 4096 tokens 65 us against 45)
      if constexpr (L == 16) {
        if (p.k < 16) {
          float* lds = area[wave] + sub * ROOM;
          if (p.top_groups == p.groups || (p.ranked && p.group_top > 1)) {
            wave_lds_order();
#pragma unroll
            for (int i = 0; i < PER; ++i) lds[lds_at(i * L + lane)] = c[i];
            wave_lds_order();
          }
          unsure |= pick_at_once<PER>(p, lane, near, c, lds, sel[slot], &done);
        }
      }
      if (!done) unsure |= pick_in_turn<float, L, PER>(p, lane, near, c, sel[slot]);
      unsure = unsure && !broken && t < p.T;
      if (t < p.T && !unsure) finish_token<F, L, PER>(p, t, lane, l, top, broken, sel[slot], base);
      again = __ballot(unsure);
    }
    // the wave's tokens whose choice 32 bits do not settle, one by one
    while (again != 0) {
      constexpr int WIDE = MOST / 64;
      const int lane = opaque_tid() & 63, first_lane = __builtin_ctzll(again);
      again &= L == 64 ? 0 : ~(0xffffull << (first_lane & 48));
      const int which = wave * TPW + first_lane / L;
      const int64_t t = (int64_t)first + t0 + which;
      float l[WIDE];
      double c[WIDE];
      load_logits<F, 64, WIDE>(p, t, lane, l);
      const float top = top_logit<64, WIDE>(p, l);
      choice_scores<double, 64, WIDE>(p, l, lane, top, c);
      if (p.top_groups < p.groups) {
        limit_groups<double, 64, WIDE>(p, lane, 0.0, (double*)area[wave], c);
        if (p.ranked) {
#pragma unroll
          for (int k = 0; k < WIDE; ++k) c[k] = c[k] > -(double)__builtin_inff() ? (double)l[k] : c[k];
        }
      }
      pick_in_turn<double, 64, WIDE>(p, lane, 0.0, c, sel[which]);
      finish_token<F, 64, WIDE>(p, t, lane, l, top, false, sel[which], base);
    }
  }
  __syncthreads();
  if (p.counts != nullptr) {
    // (a block's tokens, and so an expert's choices, number less than 2^16)
    const int words = (p.E + 1) / 2;
    for (int i = threadIdx.x; i < words; i += ROUTE_THREADS)
      p.counts[(int64_t)blockIdx.x * words + i] =
          (uint32_t)base[2 * i] | (2 * i + 1 < p.E ? (uint32_t)base[2 * i + 1] << 16 : 0u);
    return;
  }
  const int e = threadIdx.x, own = e < p.E ? base[e] : 0;
  int32_t total;
  const int32_t end = scan_threads(own, scratch, &total);
  if (e < p.E) {
    p.ends[e] = end;
    base[e] = end - own;
  }
  __syncthreads();
  for (int t0 = 0; t0 < p.T; t0 += 64) place_chunk(p, t0, load_experts(p, t0), base, mask, t0 + 64 < p.T);
  for (int i = total + (int)threadIdx.x; i < p.T * p.k; i += ROUTE_THREADS) p.tokens[i] = -1;
}

// The dispatch of many blocks' choices: each block adds up, per expert, the
// choices of all blocks and of those before it.
__global__ __launch_bounds__(ROUTE_THREADS) static void route_place(RouteParams p) {
  __shared__ uint64_t mask[ROUTE_MOST_EXPERTS];
  __shared__ int32_t base[ROUTE_MOST_EXPERTS], before[ROUTE_MOST_EXPERTS], scratch[ROUTE_THREADS / 64];
  const int b = blockIdx.x, blocks = gridDim.x;
  const int first = b * p.chunks * 64, end = min(p.T, first + p.chunks * 64);
  const HeldExperts held = load_experts(p, first);
  if (threadIdx.x < p.E) {
    base[threadIdx.x] = before[threadIdx.x] = 0;
    mask[threadIdx.x] = 0;
  }
  // Threads i, i + R, .. share the column of the experts 2 i and 2 i + 1: the rows
  // of the blocks before this one and those from its own on, 16 loads of each in
  // flight, which read zeros past their last row.  All blocks read all counts;
  // what bounds that is the instructions per count, a dot product's (unpacked and
  // added with checks of their row, 16384 tokens and 256 experts took 3.7 us of
  // 7.6; in 32 bits each 8.7 in all).
  const int words = (p.E + 1) / 2;
  int R = 64;
  while (R < words) R *= 2;
  const int i = (int)threadIdx.x & (R - 1), step = ROUTE_THREADS / R;
  uint32_t sum[2][2] = {};
  if (i < words) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const uint32_t row = (uint32_t)words * 4, rows[2] = {(uint32_t)b, (uint32_t)(blocks - b)};
    const __amdgpu_buffer_rsrc_t r[2] = {
        __builtin_amdgcn_make_buffer_rsrc(p.counts, 0, (int)(rows[0] * row), 0x00020000),
        __builtin_amdgcn_make_buffer_rsrc(p.counts + (int64_t)b * words, 0, (int)(rows[1] * row), 0x00020000)};
    uint32_t at = (uint32_t)((int)threadIdx.x / R * words + i) * 4;
    for (uint32_t n = 0; n < max(rows[0], rows[1]); n += 16 * step, at += 16 * step * row) {
      uint32_t v[2][16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < 16; ++u)
          v[h][u] = n < rows[h] ? __builtin_amdgcn_raw_buffer_load_b32(r[h], (int)(at + u * step * row), 0, 0) : 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const u16x2 x = __builtin_bit_cast(u16x2, v[h][u]);
          sum[h][0] = __builtin_amdgcn_udot2(x, (u16x2){1, 0}, sum[h][0], false);
          sum[h][1] = __builtin_amdgcn_udot2(x, (u16x2){0, 1}, sum[h][1], false);
        }
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (i < words && 2 * i + h < p.E) {
      atomicAdd(&before[2 * i + h], (int)sum[0][h]);
      atomicAdd(&base[2 * i + h], (int)sum[1][h]);
    }
  __syncthreads();
  const int e = threadIdx.x, earlier = e < p.E ? before[e] : 0, own = e < p.E ? base[e] + earlier : 0;
  int32_t total;
  const int32_t last = scan_threads(own, scratch, &total);
  if (e < p.E) {
    if (b == 0) p.ends[e] = last;
    base[e] = last - own + earlier;
  }
  __syncthreads();
  place_chunk(p, first, held, base, mask, first + 64 < end);
  for (int t0 = first + 64; t0 < end; t0 += 64) place_chunk(p, t0, load_experts(p, t0), base, mask, t0 + 64 < end);
  // the rows behind the last expert's
  for (int64_t i = (int64_t)total + b * ROUTE_THREADS + (int)threadIdx.x; i < (int64_t)p.T * p.k;
       i += blocks * ROUTE_THREADS)
    p.tokens[i] = -1;
}

// ---- the gradient ------------------------------------------------------------

struct RouteGradParams : RouteParams {
  const float* dweights;
  void* dlogits;
  int64_t ldd;
};

constexpr int ROUTE_GRAD_THREADS = 256;

// dlogits from dweights, with w_j = scale s_j (/ sum s): for the chosen experts,
// d = sum_j v_j dw_j and v = s / sum s,
//   softmax, renormalised   scale v_j (dw_j - d)
//   sigmoid, renormalised   scale v_j (1 - s_j) (dw_j - d)
//   sigmoid                 scale s_j (1 - s_j) dw_j
// and zero for the others; softmax alone: scale p_e ([e chosen] dw_j - sum_j p_j
// dw_j) for every expert.  Choices outside the experts take no part.
// Bound by instructions: 20011 tokens of 48 BF16 experts, dense, 6.0 us where its 4.8
// MB take 0.9; 16384 of 256, FP32, renormalised 10.4 (34 MB, 6.5), BF16 dense 11.8,
// of 1024 FP32 27 (134 MB, 26).  Slots beyond k are computed like those before
// it, a dense row takes a second exponential and a division a logit, and 16-bit
// rows are read and written an element a lane.
template <typename F, int L, int PER>
__global__ __launch_bounds__(ROUTE_GRAD_THREADS) void route_grad(RouteGradParams p) {
  constexpr int SLOTS = (ROUTE_MOST_K + L - 1) / L;
  const int lane = (int)threadIdx.x & (L - 1);
  const int64_t step = (int64_t)gridDim.x * (ROUTE_GRAD_THREADS / L);
  for (int64_t t0 = (int64_t)blockIdx.x * (ROUTE_GRAD_THREADS / L); t0 < p.T; t0 += step) {
    const int64_t t = t0 + (int)threadIdx.x / L;
    const bool live = t < p.T;
    float l[PER];
    load_logits<F, L, PER>(p, t, lane, l);
    const float top = top_logit<L, PER>(p, l);
    const F* row = (const F*)p.logits + (live ? t : 0) * p.ld;
    int e[SLOTS];
    float lc[SLOTS], dw[SLOTS], s[SLOTS], m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int j = i * L + lane;
      e[i] = -1;
      dw[i] = 0.0f;
      if (live && j < p.k) {
        e[i] = p.experts[t * p.k + j];
        if (e[i] >= p.E) e[i] = -1;
        if (e[i] >= 0) dw[i] = p.dweights[t * p.k + j];
      }
      lc[i] = e[i] >= 0 ? (float)row[e[i]] : -__builtin_inff();
      m = fmaxf(m, lc[i]);
    }
    m = max_lanes<L>(m);
    const ScoreBase b = score_base<L, PER>(p, l, top, m);
    float total = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      s[i] = e[i] >= 0 ? score_of(p, lc[i], b) : 0.0f;
      total += s[i];
    }
    total = sum_lanes<L>(total);
    if (!p.renorm || total == 0.0f) total = 1.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      s[i] /= total;
      d += s[i] * dw[i];
    }
    d = sum_lanes<L>(d);
    const bool dense = !p.sigmoid && !p.renorm;
    float g[SLOTS], out[PER];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      g[i] = p.scale * s[i] * (p.renorm ? dw[i] - d : dw[i]);
      if (p.sigmoid) g[i] *= 1.0f / (1.0f + expf(lc[i]));
      if (e[i] < 0) g[i] = 0.0f;
    }
    const bool any = m > -__builtin_inff();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      out[i] = dense && any ? -p.scale * d * (expf(l[i] - b.top) / b.sum) : 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      for (int j = i * L; j < min(p.k, (i + 1) * L); ++j) {
        const int from = ((int)threadIdx.x & 63 & ~(L - 1)) + j - i * L;
        const int at = __shfl(e[i], from);
        const float x = __shfl(g[i], from);
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (at == q * L + lane) out[q] += x;
      }
    if (!live) continue;
    F* dst = (F*)p.dlogits + t * p.ldd;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * L + lane < p.E) dst[i * L + lane] = (F)out[i];
  }
}

}  // namespace dg
