// route_kernel.h -- routing of tokens to experts on the MI355X (gfx950): the
// choice of every token's experts from its logits, their weights, and the
// dispatch (the order of the chosen rows by expert), with the weights'
// gradient.
//
// A token is handled by L neighbouring lanes (16, or a wave for many experts),
// PER logits a lane in registers.  The best expert is found k times: each
// lane's best, then the lanes' (lanes.h), ties to the lowest index.  The
// dispatch is a counting sort: a workgroup takes 64 tokens at a time and marks
// in a 64-bit word per expert which of them chose it (LDS atomics of an OR,
// whose order changes nothing), so that a choice's rank among them is a count of
// the bits below its token's.  The order of the rows, by expert and then by
// token, is thus fixed.
//
// Scores are compared in 32 bits where these decide.  With a bias (or sums of
// scores for groups) two candidates may lie closer together than the rounding
// errors of their scores; the token's choice is then made again in 64 bits, so
// that it does not depend on how a 32-bit exponential rounds.  Without them the
// logits themselves are compared, which is exact.
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
  int groups, group_size, top_groups, group_top;
  int chunks;          // chunks of 64 tokens per block
};

// A logit (type F: float, or a 16-bit one) as FP32.
template <typename F>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  if constexpr (sizeof(F) == 4)
    return ((const float*)row)[e];
  else
    return unpack<F>(((const uint16_t*)row)[e], 0);
}

template <typename X>
__device__ __forceinline__ X exp_of(X x) {
  if constexpr (sizeof(X) == 8)
    return exp(x);
  else
    return expf(x);
}

// The best of a token's candidates: value and index, the lowest index of equal
// values; key[] holds -inf where there is none.
template <int L, int PER, typename X>
__device__ __forceinline__ void best_of(const X (&key)[PER], int lane, X* value, int* index) {
  X m = key[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < PER; ++i)
    if (key[i] > m) {
      m = key[i];
      at = i;
    }
  const X top = max_lanes<L>(m);
  *value = top;
  *index = min_lanes<L>(m == top ? lane * PER + at : 1 << 30);
}

// What one token's lanes find out: slots j = lane, lane + L, .. of the chosen.
template <int L>
struct Chosen {
  static constexpr int SLOTS = (ROUTE_MOST_K + L - 1) / L;
  int expert[SLOTS];  // -1: none
};

// The choice in precision X.  Lane l holds experts l PER .. l PER + PER - 1 in
// l[] (-inf past E and where an expert is off).  `lds`: E values of this
// token's, for the groups.  Returns whether rounding could change it.
template <int L, int PER, typename X>
__device__ __forceinline__ bool choose(const RouteParams& p, const float (&l)[PER], int lane,
                                       X* lds, bool ranked, float top, Chosen<L>* out) {
  const X NONE = -(X)__builtin_inff();
  X c[PER];
  X smax = 1;
  if (ranked && p.group_top == 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i];
  } else {
    X sum = 0;
    if (!p.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = exp_of<X>((X)l[i] - (X)top);
        sum += c[i];
      }
      sum = sum_lanes<L>(sum);
      smax = 1 / sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = c[i] / sum;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = 1 / (1 + exp_of<X>(-(X)l[i]));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (p.bias != nullptr && e < p.E) c[i] += (X)p.bias[e];
      if (!(l[i] > -__builtin_inff()) || !(c[i] > NONE)) c[i] = NONE;
    }
  }
  const bool exact = (ranked && (p.group_top == 1 || p.top_groups == p.groups)) || sizeof(X) == 8;
  // Errors of c in 32 bits: a logistic's 2^-22; a softmax's 2^-18 of its size (its
  // sum's, above all); the sum with the bias 2^-24 |c|.  A group's value has two of
  // each, a difference of two values twice that.
  const X near = (p.sigmoid ? (X)0x1p-19 : smax * (X)0x1p-15);
  bool unsure = false;
  auto close = [&](X a, X b, X size) {
    // (a difference that is no number counts as close)
    if (exact || !(a > NONE) || !(b > NONE)) return;
    if (!(a - b > near + (X)0x1p-20 * size)) unsure = true;
  };
  if (p.top_groups < p.groups) {
    // a group's value from LDS, a group per lane
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < p.E) lds[lane * PER + i] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    constexpr int GS = (ROUTE_MOST_GROUPS + L - 1) / L;
    X value[GS], size = 0;
#pragma unroll
    for (int g0 = 0; g0 < GS; ++g0) {
      const int g = lane * GS + g0;
      X first = NONE, second = NONE;
      if (g < p.groups)
        for (int i = 0; i < p.group_size; ++i) {
          const X x = lds[g * p.group_size + i];
          if (x > first) {
            second = first;
            first = x;
          } else if (x > second) {
            second = x;
          }
        }
      const bool two = p.group_top > 1 && second > NONE;
      value[g0] = two ? first + second : first;
      if (first > NONE) size = fmax(size, fmax(fabs(first), two ? fabs(second) : (X)0));
    }
    size = max_lanes<L>(size);
    uint64_t stays = 0;
    X before = 0;
    for (int n = 0; n <= p.top_groups; ++n) {
      X v;
      int g;
      best_of<L, GS>(value, lane, &v, &g);
      if (n == p.top_groups) {
        close(before, v, size);
        break;
      }
      before = v;
      if (!(v > NONE)) break;
      stays |= 1ull << g;
#pragma unroll
      for (int g0 = 0; g0 < GS; ++g0)
        if (lane * GS + g0 == g) value[g0] = NONE;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      if (e < p.E && !(stays >> (e / p.group_size) & 1)) c[i] = NONE;
    }
    if (ranked && p.group_top > 1) {
      // (sums of scores chose the groups; within them the logits rank)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (c[i] > NONE) c[i] = l[i];
    }
  } else if (ranked && p.group_top > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i];
  }
#pragma unroll
  for (int s = 0; s < Chosen<L>::SLOTS; ++s) out->expert[s] = -1;
  X before = 0;
  // (one round more than choices, where the next candidate's distance counts)
  const int rounds = ranked || sizeof(X) == 8 ? p.k : p.k + 1;
  for (int j = 0; j < rounds; ++j) {
    X v;
    int e;
    best_of<L, PER>(c, lane, &v, &e);
    if (!ranked && j > 0) close(before, v, fmax(fabs(before), fabs(v)));
    before = v;
    if (j == p.k) break;
    if (v > NONE) {
#pragma unroll
      for (int s = 0; s < Chosen<L>::SLOTS; ++s)
        if (j == s * L + lane) out->expert[s] = e;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (lane * PER + i == e) c[i] = NONE;
    }
  }
  return unsure;
}

// The order of the chosen rows, for the 64 tokens from t0 on (as many as there
// are), from their experts in memory: each choice's place, and its token there.
// base[e]: the place of the first of them that chose e; mask: E words.  Ends
// with a barrier; base has moved on.
__device__ __forceinline__ void place_chunk(const RouteParams& p, int t0, int32_t* base,
                                            uint64_t* mask) {
  const int n = min(64, p.T - t0) * p.k;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)t0 * p.k;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = p.experts[s0 + i];
    if (e >= 0) atomicOr((unsigned long long*)&mask[e], 1ull << (i / p.k));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = p.experts[s0 + i], t = i / p.k;
    int at = -1;
    if (e >= 0) {
      at = base[e] + __popcll(mask[e] & ((1ull << t) - 1));
      p.tokens[at] = t0 + t;
    }
    p.places[s0 + i] = at;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) base[e] += __popcll(mask[e]);
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

// One token's logits: lane l's are l PER .. l PER + PER - 1; -inf past E (and
// everywhere for a token that there is not).
template <typename F, int PER>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&l)[PER]) {
  const int e0 = lane * PER;
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = -__builtin_inff();
  if (t >= p.T || e0 >= p.E) return;
  if constexpr (sizeof(F) == 4) {
    typedef f32x4 f32x4_any __attribute__((aligned(4)));
    const float* row = (const float*)p.logits + t * p.ld + e0;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      if (e0 + i + 4 <= p.E) {
        const f32x4 x = *(const f32x4_any*)(row + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) l[i + k] = x[k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (e0 + i + k < p.E) l[i + k] = row[i + k];
      }
    }
  } else {
    constexpr int W = PER < 8 ? 2 : 4;
    const uint16_t* row = (const uint16_t*)p.logits + t * p.ld;
#pragma unroll
    for (int i = 0; i < PER; i += 2 * W) {
      uint32_t x[W];
      if (e0 + i >= p.E) break;
      load_row<W>(row, e0 + i, p.E, x);
#pragma unroll
      for (int k = 0; k < 2 * W; ++k)
        if (e0 + i + k < p.E) l[i + k] = unpack<F>(x[k >> 1], k & 1);
    }
  }
}

// The largest of a token's logits, and whether one is NaN or +inf.
template <int L, int PER>
__device__ __forceinline__ bool broken_row(const float (&l)[PER], float* top) {
  float m = l[0];
  int bad = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    bad |= !(l[i] < __builtin_inff());
    m = l[i] > m ? l[i] : m;
  }
  m = max_lanes<L>(m);
  *top = m > -__builtin_inff() ? m : 0.0f;
  return reduce_lanes<L>(bad, [](int a, int b) { return a | b; }) != 0;
}

// The scores of up to L chosen logits, one a lane (on: whether there is one),
// or several in turn: a common factor is left out of them where they will be
// divided by their sum, so that none underflows beside larger ones.
struct ScoreBase {
  float top;  // what the factor is made of
  float sum;  // the softmax's sum over all experts, or 1
};
__device__ __forceinline__ float score_of(const RouteParams& p, float l, const ScoreBase& b) {
  if (!p.sigmoid) return expf(l - b.top) / b.sum;
  if (l > 0.0f) return 1.0f / (1.0f + expf(-l));
  return expf(l - b.top) / (1.0f + expf(l));
}

// (sum over all experts of a row: every lane's, then the lanes')
template <int L, int PER>
__device__ __forceinline__ float softmax_sum(const float (&l)[PER], float top) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) s += expf(l[i] - top);
  return sum_lanes<L>(s);
}

template <int L, int PER>
__device__ __forceinline__ ScoreBase score_base(const RouteParams& p, const float (&l)[PER], float top,
                                                float top_chosen) {
  ScoreBase b = {0.0f, 1.0f};
  if (p.renorm) {
    b.top = p.sigmoid ? fminf(top_chosen, 0.0f) : top_chosen;
  } else if (!p.sigmoid) {
    b.top = top;
    b.sum = softmax_sum<L, PER>(l, top);
  }
  return b;
}

// The choice: a block takes `chunks` times 64 tokens.  A lone block also makes
// the dispatch; otherwise each leaves its choices per expert in counts, for
// route_place.
template <typename F, int L, int PER>
__global__ __launch_bounds__(ROUTE_THREADS) void route_choose(RouteParams p) {
  constexpr int TPW = 64 / L;  // tokens per wave
  constexpr int AT_ONCE = ROUTE_THREADS / L, MOST = L * PER;
  // a wave's scores, by token (a pair of them holds one token's in 64 bits)
  __shared__ __attribute__((aligned(16))) float area[ROUTE_THREADS / 64][(TPW < 2 ? 2 : TPW) * MOST];
  __shared__ uint64_t mask[MOST];
  __shared__ int32_t base[MOST], scratch[ROUTE_THREADS / 64];
  const int lane = (int)threadIdx.x & (L - 1), wave = (int)threadIdx.x >> 6;
  const int sub = ((int)threadIdx.x & 63) / L;
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) base[e] = 0;
  __syncthreads();
  const int first = (int)blockIdx.x * p.chunks * 64, last = min(p.T - first, p.chunks * 64);
  const bool ranked = p.bias == nullptr;
  for (int t0 = 0; t0 < last; t0 += AT_ONCE) {
    const int64_t t = (int64_t)first + t0 + (int)threadIdx.x / L;
    float l[PER], top;
    load_logits<F, PER>(p, t, lane, l);
    const bool broken = broken_row<L, PER>(l, &top);
    if (broken) {
#pragma unroll
      for (int i = 0; i < PER; ++i) l[i] = -__builtin_inff();
      top = 0.0f;
    }
    Chosen<L> ch;
    const bool unsure = choose<L, PER, float>(p, l, lane, area[wave] + sub * MOST, ranked, top, &ch);
    if (__ballot(unsure) != 0) {
      for (int q = 0; q < TPW; ++q)
        if (unsure && q == sub)
          choose<L, PER, double>(p, l, lane, (double*)area[wave], ranked, top, &ch);
    }
    // the weights, from the chosen logits
    float lc[Chosen<L>::SLOTS], m = -__builtin_inff();
    const void* row = (const char*)p.logits + (t < p.T ? t : 0) * p.ld * (int)sizeof(F);
#pragma unroll
    for (int s = 0; s < Chosen<L>::SLOTS; ++s) {
      lc[s] = ch.expert[s] >= 0 ? logit_at<F>(row, ch.expert[s]) : -__builtin_inff();
      m = fmaxf(m, lc[s]);
    }
    m = max_lanes<L>(m);
    const ScoreBase b = score_base<L, PER>(p, l, top, m);
    float total = 0.0f;
#pragma unroll
    for (int s = 0; s < Chosen<L>::SLOTS; ++s) {
      lc[s] = ch.expert[s] >= 0 ? score_of(p, lc[s], b) : 0.0f;
      total += lc[s];
    }
    total = sum_lanes<L>(total);
    if (!p.renorm || total == 0.0f) total = 1.0f;
    if (t < p.T) {
#pragma unroll
      for (int s = 0; s < Chosen<L>::SLOTS; ++s) {
        const int j = s * L + lane;
        if (j >= p.k) break;
        p.weights[t * p.k + j] = broken ? __builtin_nanf("") : lc[s] / total * p.scale;
        p.experts[t * p.k + j] = ch.expert[s];
        if (ch.expert[s] >= 0) atomicAdd(&base[ch.expert[s]], 1);
      }
    }
  }
  __syncthreads();
  if (p.counts != nullptr) {
    for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS)
      p.counts[(int64_t)blockIdx.x * p.E + e] = base[e];
    return;
  }
  const int total = scan_experts(base, p.E, scratch);
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) p.ends[e] = e + 1 < p.E ? base[e + 1] : total;
  __syncthreads();
  for (int t0 = 0; t0 < p.T; t0 += 64) place_chunk(p, t0, base, mask);
  for (int i = total + (int)threadIdx.x; i < p.T * p.k; i += ROUTE_THREADS) p.tokens[i] = -1;
}

// The dispatch of many blocks' choices: each block adds up, per expert, the
// choices of all blocks and of those before it.
__global__ __launch_bounds__(ROUTE_THREADS) static void route_place(RouteParams p) {
  __shared__ uint64_t mask[ROUTE_MOST_EXPERTS];
  __shared__ int32_t base[ROUTE_MOST_EXPERTS], before[ROUTE_MOST_EXPERTS], scratch[ROUTE_THREADS / 64];
  const int b = blockIdx.x, blocks = gridDim.x;
  for (int e = threadIdx.x; e < p.E; e += ROUTE_THREADS) base[e] = before[e] = 0;
  __syncthreads();
  // threads e, e + R, .. share expert e's column of the counts
  int R = 64;
  while (R < p.E) R *= 2;
  const int e = (int)threadIdx.x & (R - 1), step = ROUTE_THREADS / R;
  if (e < p.E) {
    int all = 0, mine = 0;
    const int32_t* c = p.counts + e;
    for (int i0 = (int)threadIdx.x / R; i0 < blocks; i0 += 8 * step) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i0 + u * step < blocks ? c[(int64_t)(i0 + u * step) * p.E] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
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
  const int first = b * p.chunks * 64, end = min(p.T, first + p.chunks * 64);
  for (int t0 = first; t0 < end; t0 += 64) place_chunk(p, t0, base, mask);
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
  constexpr int SLOTS = Chosen<L>::SLOTS;
  const int lane = (int)threadIdx.x & (L - 1);
  const int64_t step = (int64_t)gridDim.x * (ROUTE_GRAD_THREADS / L);
  for (int64_t t0 = (int64_t)blockIdx.x * (ROUTE_GRAD_THREADS / L); t0 < p.T; t0 += step) {
    const int64_t t = t0 + (int)threadIdx.x / L;
    const bool live = t < p.T;
    float l[PER], top;
    load_logits<F, PER>(p, t, lane, l);
    broken_row<L, PER>(l, &top);
    const void* row = (const char*)p.logits + (live ? t : 0) * p.ld * (int)sizeof(F);
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
      lc[i] = e[i] >= 0 ? logit_at<F>(row, e[i]) : -__builtin_inff();
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
        const int at = __shfl(e[i], from) - lane * PER;
        const float x = __shfl(g[i], from);
#pragma unroll
        for (int q = 0; q < PER; ++q)
          if (at == q) out[q] += x;
      }
    const int e0 = lane * PER;
    if (!live || e0 >= p.E) continue;
    if constexpr (sizeof(F) == 4) {
      float* dst = (float*)p.dlogits + t * p.ldd + e0;
      typedef f32x4 f32x4_any __attribute__((aligned(4)));
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        if (e0 + i + 4 <= p.E) {
          *(f32x4_any*)(dst + i) = (f32x4){out[i], out[i + 1], out[i + 2], out[i + 3]};
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (e0 + i + k < p.E) dst[i + k] = out[i + k];
        }
      }
    } else {
      constexpr int W = PER < 8 ? 2 : 4;
      uint16_t* dst = (uint16_t*)p.dlogits + t * p.ldd;
#pragma unroll
      for (int i = 0; i < PER; i += 2 * W) {
        if (e0 + i >= p.E) break;
        uint32_t o[W];
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = pack2<F>(out[i + 2 * k], out[i + 2 * k + 1]);
        store_row<W>(dst, e0 + i, p.E, o);
      }
    }
  }
}

}  // namespace dg
