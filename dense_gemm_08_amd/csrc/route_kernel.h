// route_kernel.h -- routing of tokens to experts on the MI355X (gfx950): the
// choice of every token's experts from its logits, their weights, and the
// dispatch (the order of the chosen rows by expert), with the weights'
// gradient.
//
// A token is handled by L neighbouring lanes (16, or a wave for many experts),
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
  int32_t* counts;     // choices per block and expert (null: one block)
  int64_t ld;
  int T, E, k;
  int sigmoid, renorm;
  float scale;
  int ranked;          // no bias: the logits rank the experts
  int groups, group_size, top_groups, group_top;
  int group_lanes;     // lanes that look for a group's best: a power of two
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
// Returns by how much two of them have to differ, next to 2^-22 of their size,
// for their order to be sure (sums of two: by twice as much): in 32 bits a
// logistic's error is below 2^-22, a softmax's 2^-18 of the largest (the sum's,
// above all), the bias's sum rounds by 2^-24, and a difference has two of each.
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
  X near = (X)0x1p-20;
  if (!p.sigmoid) {
    X sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (FAST)
        c[i] = __builtin_amdgcn_exp2f((l[i] - top) * L2E);
      else
        c[i] = exp((X)l[i] - (X)top);
      sum += c[i];
      if constexpr (!FAST) fence();  // (one after the other: they take many registers)
    }
    const X part = 1 / sum_lanes<L>(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] *= part;
    near = part * (X)0x1p-16;
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
      fence();
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
// which the lanes compare and combine in fewer instructions; and back.
constexpr int KEY_NONE = (int)0x807fffff;  // -inf
constexpr int KEY_PAD = -0x7fffffff;       // below all values
__device__ __forceinline__ int key_of(float x) {
  const int b = __builtin_bit_cast(int, x + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int key) {
  return __builtin_bit_cast(float, key ^ ((key >> 31) & 0x7fffffff));
}

// How many of a row's 16 keys go before this lane's: the larger ones, and of
// equal ones those of lower lanes.
__device__ __forceinline__ int rank_in_row(int key) {
  const int lane = (int)threadIdx.x & 15;
  int rank = 0;
  for_others([&](auto n) {
    constexpr int N = decltype(n)::value;
    // (the key comes from lane - N, a lower one unless that counts around)
    rank += rotated<N>(key) > (lane >= N ? key - 1 : key) ? 1 : 0;
  });
  return rank;
}
// The 16 bits of a wave's ballot that are this lane's row's.
__device__ __forceinline__ uint32_t row_bits(uint64_t ballot) {
  const int lane = (int)threadIdx.x & 63;
  const uint32_t half = lane < 32 ? (uint32_t)ballot : (uint32_t)(ballot >> 32);
  return lane & 16 ? half >> 16 : half & 0xffffu;
}

// Whether a, the larger, is not surely larger than b; size: that of what they
// were summed from.
template <typename X>
__device__ __forceinline__ bool too_close(X a, X b, X near, X size) {
  if (sizeof(X) == 8 || !(b > -(X)__builtin_inff())) return false;
  return !(a - b > near + (X)0x1p-22 * size);  // (so is a difference that is no number)
}

// Takes the experts outside the best groups from c.  `lds`: E values of this
// token's.  Returns whether rounding could change that.
template <typename X, int L, int PER>
__device__ __forceinline__ bool limit_groups(const RouteParams& p, int lane, X near, X* lds, X (&c)[PER]) {
  const X NONE = -(X)__builtin_inff();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * L + lane < p.E) lds[i * L + lane] = c[i];
  wave_lds_order();
  // A group's two best, found by `share` neighbouring lanes (up to 16, a power
  // of two) where there are no more groups than lanes; else several groups a
  // lane.
  constexpr int GS = (ROUTE_MOST_GROUPS + L - 1) / L;
  X value[GS], size = 0;
  const int share = p.group_lanes;
#pragma unroll
  for (int n = 0; n < GS; ++n) {
    const int g = n * L + lane / share;
    X first = NONE, second = NONE;
    if (g < p.groups) {
      const X* from = lds + g * p.group_size;
#pragma unroll 4
      for (int i = lane & (share - 1); i < p.group_size; i += share) {
        const X x = from[i];
        second = fmax(second, fmin(first, x));
        first = fmax(first, x);
      }
    }
    auto join = [&](X f, X s) {
      second = fmax(fmin(first, f), fmax(second, s));
      first = fmax(first, f);
    };
    if (share > 1) join(dpp_move<0xB1>(first), dpp_move<0xB1>(second));
    if (share > 2) join(dpp_move<0x4E>(first), dpp_move<0x4E>(second));
    if (share > 4) join(dpp_move<0x141>(first), dpp_move<0x141>(second));
    if (share > 8) join(dpp_move<0x140>(first), dpp_move<0x140>(second));
    const bool two = p.group_top > 1 && second > NONE;
    value[n] = two ? first + second : first;
    if (first > NONE) size = fmax(size, fmax(fabs(first), two ? fabs(second) : (X)0));
    if (share > 1) break;
  }
  bool unsure = false;
  if (p.ranked && p.group_top == 1) near = size = 0;
  const bool exact = p.ranked && p.group_top == 1;
  size = max_lanes<L>(size);
  uint64_t stays = 0;  // bit (group * share)
  if (sizeof(X) == 4 && L == 16 && p.groups <= 16) {
    // the groups ranked all at once, each by the first of its lanes
    const bool first = (lane & (share - 1)) == 0;
    const int key = first ? key_of((float)value[0]) : KEY_PAD;
    const int rank = rank_in_row(key);
    const bool stay = first && key > KEY_NONE && rank < p.top_groups;
    stays = row_bits(__ballot(stay));
    const int least = min_lanes<16>(stay ? key : 0x7fffffff);
    const int next = max_lanes<16>(stay ? KEY_PAD : key);
    if (!exact && next > KEY_NONE) unsure = too_close((X)value_of(least), (X)value_of(next), 2 * near, 4 * size);
  } else {
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
      const X best = max_lanes<L>(m);
      if (!(best > NONE)) break;
      if (n == p.top_groups) {
        unsure = !exact && too_close(least, best, 2 * near, 4 * size);
        break;
      }
      least = best;
      const int g = min_lanes<L>(m == best ? at : 1 << 30);
      stays |= 1ull << (g * share & 63);
#pragma unroll
      for (int i = 0; i < GS; ++i)
        if ((share > 1 ? lane / share : i * L + lane) == g) value[i] = NONE;
    }
  }
  auto keep = [&](int i, int g) {
    const int bit = g * share & 63;
    const bool stay = (bit < 32 ? (uint32_t)stays : (uint32_t)(stays >> 32)) >> (bit & 31) & 1;
    if (!stay) c[i] = NONE;
  };
  if (p.group_size % L == 0) {  // (an element's group is the same one in all lanes)
#pragma unroll
    for (int i = 0; i < PER; ++i) keep(i, i * L * p.group_inverse >> 20);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) keep(i, (i * L + lane) * p.group_inverse >> 20);
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
    const X best = max_lanes<L>(m);
    if (!p.ranked && j > 0) unsure |= too_close(before, best, near, (X)fmax(fabs(before), fabs(best)));
    before = best;
    if (j == p.k) break;
    const int e = min_lanes<L>(m == best ? at * L + lane : 1 << 30);
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
// others are not (256 experts, 8 chosen: 14 expected).  These candidates are
// gathered in LDS in the order of their index, two a lane at most, and ranked by
// comparing each with all: about 350 instructions where 9 maxima in turn take
// about 900.  `lds`: 64 words of this token's.  *done is false, for the whole
// wave, if some token has more than 32.
template <int PER>
__device__ __forceinline__ bool pick_at_once(const RouteParams& p, int lane, float near, const float (&c)[PER],
                                             float* lds, int* sel, bool* done) {
  int key[PER], m = KEY_NONE;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = key_of(c[i]);
    m = max(m, key[i]);
  }
  const int limit = max(min_lanes<16>(rank_in_row(m) <= p.k ? m : 0x7fffffff), KEY_NONE + 1);
  u32x2* cand = (u32x2*)lds;  // (key, expert)
  cand[lane] = cand[lane + 16] = (u32x2){(uint32_t)KEY_PAD, 0u};
  wave_lds_order();
  const uint32_t below = (1u << lane) - 1;
  int total = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool is = key[i] >= limit;
    const uint32_t row = row_bits(__ballot(is));
    const int at = total + __popc(row & below);
    if (is && at < 32) cand[at] = (u32x2){(uint32_t)key[i], (uint32_t)(i * 16 + lane)};
    total += __popc(row);
  }
  *done = __ballot(total > 32) == 0;
  if (!*done) return false;
  wave_lds_order();
  const u32x2 x = cand[lane], y = cand[lane + 16];
  const int a = (int)x[0], b = (int)y[0];
  int rank_a = rank_in_row(a), rank_b = 32;
  if (__ballot(total > 16) != 0) {
    // (all of the second sixteen come after the first in the order of experts)
    rank_a += b > a ? 1 : 0;
    rank_b = rank_in_row(b) + (a >= b ? 1 : 0);
    for_others([&](auto n) {
      constexpr int N = decltype(n)::value;
      rank_a += rotated<N>(b) > a ? 1 : 0;
      rank_b += rotated<N>(a) >= b ? 1 : 0;
    });
  }
  // in order: the experts to sel, the keys (of which the next one counts) to lds
  int* sorted = (int*)lds;
  wave_lds_order();
  sorted[lane] = KEY_NONE;
  if (lane < p.k) sel[lane] = -1;
  wave_lds_order();
  if (a > KEY_NONE && rank_a <= p.k) {
    sorted[rank_a] = a;
    if (rank_a < p.k) sel[rank_a] = (int)x[1];
  }
  if (b > KEY_NONE && rank_b <= p.k) {
    sorted[rank_b] = b;
    if (rank_b < p.k) sel[rank_b] = (int)y[1];
  }
  wave_lds_order();
  if (p.ranked) return false;
  const float v = value_of(sorted[lane]), w = value_of(sorted[lane < 15 ? lane + 1 : 15]);
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
// last at the end; mask: E words of zeros, left so.
__device__ __forceinline__ void place_chunk(const RouteParams& p, int t0, const HeldExperts& h, int32_t* base,
                                            uint64_t* mask) {
  const int n = min(64, p.T - t0) * p.k;
  int t[HELD];
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    const int i = u * ROUTE_THREADS + (int)threadIdx.x;
    t[u] = (int)((uint32_t)(i * p.k_inverse) >> 20);
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
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) {
    base[e] += __popcll(mask[e]);
    mask[e] = 0;
  }
  __syncthreads();
}

// The running sums of x[0 .. E) over the block's threads, exclusive, written
// over x; the total is returned.  scratch: one value per wave.
__device__ __forceinline__ int32_t scan_experts(int32_t* x, int E, int32_t* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int32_t v = e < E ? x[e] : 0;
    int32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int32_t y = __shfl_up(s, d);
      if (lane >= d) s += y;
    }
    if (lane == 63) scratch[wave] = s;
    __syncthreads();
    int32_t before = carry;
    for (int w = 0; w < waves; ++w) {
      if (w < wave) before += scratch[w];
      carry += scratch[w];
    }
    if (e < E) x[e] = before + s - v;
    __syncthreads();
  }
  return carry;
}

// The choice: a block takes `chunks` times 64 tokens.  A lone block also makes
// the dispatch; otherwise each leaves its choices per expert in counts, for
// route_place.
template <typename F, int L, int PER>
__global__ __launch_bounds__(ROUTE_THREADS) void route_choose(RouteParams p) {
  constexpr int TPW = 64 / L, WAVES_RT = ROUTE_THREADS / 64;
  constexpr int AT_ONCE = ROUTE_THREADS / L, MOST = L * PER;
  // a wave's scores, by token (in 64 bits one token's)
  __shared__ __attribute__((aligned(16))) float area[WAVES_RT][(TPW < 2 ? 2 : TPW) * MOST];
  __shared__ int sel[AT_ONCE][ROUTE_MOST_K];  // the chosen, in order
  __shared__ int again[AT_ONCE], agains;
  __shared__ uint64_t mask[MOST];
  __shared__ int32_t base[MOST], scratch[WAVES_RT];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) {
    base[e] = 0;
    mask[e] = 0;
  }
  if (threadIdx.x == 0) agains = 0;
  __syncthreads();
  const int first = (int)blockIdx.x * p.chunks * 64, tokens = min(p.T - first, p.chunks * 64);
  for (int t0 = 0; t0 < tokens; t0 += AT_ONCE) {
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
        unsure = limit_groups<float, L, PER>(p, lane, near, area[wave] + sub * MOST, c);
        if (p.ranked && p.group_top > 1) {
          // (sums of scores chose the groups; within them the logits rank)
#pragma unroll
          for (int i = 0; i < PER; ++i) c[i] = c[i] > -__builtin_inff() ? l[i] : c[i];
        }
      }
      if constexpr (L == 16) {
        if (p.k < 16)
          unsure |= pick_at_once<PER>(p, lane, near, c, area[wave] + sub * MOST, sel[slot], &done);
      }
      if (!done) unsure |= pick_in_turn<float, L, PER>(p, lane, near, c, sel[slot]);
      if (t < p.T) {
        if (broken || !unsure)
          finish_token<F, L, PER>(p, t, lane, l, top, broken, sel[slot], base);
        else if (lane == 0)
          again[atomicAdd(&agains, 1)] = slot;
      }
    }
    __syncthreads();
    // the tokens whose choice 32 bits do not settle, a wave each
    for (int i = wave; i < agains; i += WAVES_RT) {
      constexpr int WIDE = MOST / 64;
      const int l64 = opaque_tid() & 63, which = again[i];
      const int64_t t = (int64_t)first + t0 + which;
      float l[WIDE];
      double c[WIDE];
      load_logits<F, 64, WIDE>(p, t, l64, l);
      const float top = top_logit<64, WIDE>(p, l);
      choice_scores<double, 64, WIDE>(p, l, l64, top, c);
      if (p.top_groups < p.groups) {
        limit_groups<double, 64, WIDE>(p, l64, 0.0, (double*)area[wave], c);
        if (p.ranked) {
#pragma unroll
          for (int k = 0; k < WIDE; ++k) c[k] = c[k] > -(double)__builtin_inff() ? (double)l[k] : c[k];
        }
      }
      pick_in_turn<double, 64, WIDE>(p, l64, 0.0, c, sel[which]);
      finish_token<F, 64, WIDE>(p, t, l64, l, top, false, sel[which], base);
    }
    __syncthreads();
    if (threadIdx.x == 0) agains = 0;
    __syncthreads();
  }
  if (p.counts != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS)
      p.counts[(int64_t)blockIdx.x * p.E + e] = base[e];
    return;
  }
  const int total = scan_experts(base, p.E, scratch);
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) p.ends[e] = e + 1 < p.E ? base[e + 1] : total;
  __syncthreads();
  for (int t0 = 0; t0 < p.T; t0 += 64) place_chunk(p, t0, load_experts(p, t0), base, mask);
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
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) {
    base[e] = before[e] = 0;
    mask[e] = 0;
  }
  __syncthreads();
  // threads e, e + R, .. share expert e's column of the counts, 16 loads in
  // flight
  int R = 64;
  while (R < p.E) R *= 2;
  const int e = (int)threadIdx.x & (R - 1), step = ROUTE_THREADS / R;
  if (e < p.E) {
    int all = 0, mine = 0;
    for (int i0 = (int)threadIdx.x / R; i0 < blocks; i0 += 16 * step) {
      const int32_t* c = p.counts + (int64_t)i0 * p.E + e;
      int v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = i0 + u * step < blocks ? c[u * step * p.E] : 0;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        all += v[u];
        mine += i0 + u * step < b ? v[u] : 0;
      }
    }
    atomicAdd(&base[e], all);
    atomicAdd(&before[e], mine);
  }
  __syncthreads();
  const int total = scan_experts(base, p.E, scratch);
  if (b == 0)
    for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) p.ends[i] = i + 1 < p.E ? base[i + 1] : total;
  __syncthreads();
  for (int i = threadIdx.x; i < p.E; i += ROUTE_THREADS) base[i] += before[i];
  __syncthreads();
  place_chunk(p, first, held, base, mask);
  for (int t0 = first + 64; t0 < end; t0 += 64) place_chunk(p, t0, load_experts(p, t0), base, mask);
  // the rows behind the last expert's
  for (int i = total + b * ROUTE_THREADS + (int)threadIdx.x; i < p.T * p.k; i += blocks * ROUTE_THREADS)
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
