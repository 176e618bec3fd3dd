// plan_experts.cpp -- argument checks and plans of what stands around an expert
// layer's products, and of the int8 products (plan_experts.h).  Plain C++ with
// no device code, so it also builds with the host sanitizers.
#include "plan_experts.h"

#include <initializer_list>

namespace dg {

namespace {

constexpr size_t kMaxBytes = (size_t)1 << 62;

bool valid_fmt(int fmt) { return fmt == DENSE_GEMM_F16 || fmt == DENSE_GEMM_BF16; }

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// A matrix of 16-bit elements that a call needs.
dense_gemm_status check_rows(const void* p, int64_t ld, int64_t cols) {
  if (p == nullptr) return DENSE_GEMM_NULL_PTR;
  if (ld < cols) return DENSE_GEMM_BAD_LD;
  if (ld >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  return aligned(p, 2) ? DENSE_GEMM_OK : DENSE_GEMM_MISALIGNED;
}

// An array of 4-byte values that a call needs (null: whether it may be).
dense_gemm_status check_words(const void* p, bool may_be_null) {
  if (p == nullptr) return may_be_null ? DENSE_GEMM_OK : DENSE_GEMM_NULL_PTR;
  return aligned(p, 4) ? DENSE_GEMM_OK : DENSE_GEMM_MISALIGNED;
}

dense_gemm_status first_of(dense_gemm_status a, dense_gemm_status b) {
  return a != DENSE_GEMM_OK ? a : b;
}

// What the two routing calls have in common.
dense_gemm_status check_routing(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                int64_t ldl, const dense_gemm_routing* r) {
  if ((!valid_fmt(fmt) && fmt != DENSE_GEMM_F32) || r == nullptr) return DENSE_GEMM_BAD_ARG;
  if (T < 0 || E < 0 || k < 0) return DENSE_GEMM_INVALID_DIM;
  if (E == 0 || k == 0 || k > E) return DENSE_GEMM_BAD_ARG;
  if (E > ROUTE_MOST_EXPERTS || k > ROUTE_MOST_K || T > kRouteMostRows / k) return DENSE_GEMM_TOO_LARGE;
  if ((r->score != DENSE_GEMM_SOFTMAX && r->score != DENSE_GEMM_SIGMOID) || (r->renorm & ~1) != 0)
    return DENSE_GEMM_BAD_ARG;
  if (T == 0) return DENSE_GEMM_OK;
  if (logits == nullptr) return DENSE_GEMM_NULL_PTR;
  if (ldl < E) return DENSE_GEMM_BAD_LD;
  if (ldl >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
  return aligned(logits, fmt == DENSE_GEMM_F32 ? 4 : 2) ? DENSE_GEMM_OK : DENSE_GEMM_MISALIGNED;
}

}  // namespace

dense_gemm_status route_validate(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                 int64_t ldl, const dense_gemm_routing* r, const void* weights,
                                 const void* experts, const void* places, const void* ends,
                                 const void* tokens) {
  const dense_gemm_status st = check_routing(fmt, T, E, k, logits, ldl, r);
  if (st != DENSE_GEMM_OK) return st;
  if (r->groups < 1 || r->groups > ROUTE_MOST_GROUPS || E % r->groups != 0 || r->top_groups < 1 ||
      r->top_groups > r->groups || r->group_top < 1 || r->group_top > 2)
    return DENSE_GEMM_BAD_ARG;
  // (every token could have k experts)
  if (k > E / r->groups * r->top_groups) return DENSE_GEMM_BAD_ARG;
  dense_gemm_status a = check_words(r->bias, true);
  a = first_of(a, check_words(ends, false));
  if (T == 0) return a;
  for (const void* p : {weights, experts, places, tokens}) a = first_of(a, check_words(p, false));
  return a;
}

dense_gemm_status route_grad_validate(int fmt, int64_t T, int64_t E, int64_t k, const void* logits,
                                      int64_t ldl, const dense_gemm_routing* r, const void* experts,
                                      const void* dweights, const void* dlogits, int64_t ldd,
                                      bool* done) {
  *done = true;
  const dense_gemm_status st = check_routing(fmt, T, E, k, logits, ldl, r);
  if (st != DENSE_GEMM_OK || T == 0) return st;
  dense_gemm_status a = check_words(experts, false);
  a = first_of(a, check_words(dweights, false));
  a = first_of(a, check_rows(dlogits, ldd, E));
  if (a == DENSE_GEMM_OK && !aligned(dlogits, fmt == DENSE_GEMM_F32 ? 4 : 2)) a = DENSE_GEMM_MISALIGNED;
  *done = a != DENSE_GEMM_OK;
  return a;
}

// Up to ROUTE_ALONE tokens one block makes the choice and the dispatch; beyond,
// blocks of 64 tokens (more where they would number over ROUTE_BLOCKS: every
// block of the second launch reads all blocks' counts; but less than 2^16, which
// those hold).  64 are the bits of the word that ranks an expert's tokens, and give
// each CU a block at 16384 tokens.
// Measured (logistic, bias, 8 chosen, FP32; us on the GPU), one block against two
// launches: 64 experts, 80 tokens 10.6 and 10.2, 128 11.3 and 10.2, 256 19.7 and
// 10.4; 256 experts 14.9 and 12.6, 16.6 and 13.2, 33 and 17; 1024 experts 56 and 49,
// 87 and 49, 169 and 49.  What one block saves is the host's: 11.5 us a call where
// two launches and their workspace take 15.8, so from 65 to 128 tokens it is the
// faster of the two for 64 experts in eager calls, about even for 256, and the
// slower for 1024.
// ROUTE_BLOCKS 256, 512 and 1024 (BF16): 65536 tokens of 64 experts 29, 32 and 44, of
// 256 42, 48 and 70, of 1024 296, 317 and 394; 131072 of 256 72, 76 and 98; 32768 of
// 256, which 512 leaves at 64 a block, 27.5 and 33.8.
constexpr int64_t ROUTE_ALONE = 128, ROUTE_BLOCKS = 512, ROUTE_CHUNKS = 1000;
RoutePlan route_plan(int64_t T, int64_t E) {
  RoutePlan p;
  const int64_t chunks = (T + 63) / 64;
  if (T <= ROUTE_ALONE) {
    p.chunks = chunks;
    p.blocks = 1;
    p.bytes = 0;
    return p;
  }
  p.chunks = (chunks + ROUTE_BLOCKS - 1) / ROUTE_BLOCKS;
  if (p.chunks > ROUTE_CHUNKS) p.chunks = ROUTE_CHUNKS;
  p.blocks = (chunks + p.chunks - 1) / p.chunks;
  p.bytes = (size_t)((p.blocks * ((E + 1) / 2) * 4 + 255) & ~(int64_t)255);
  return p;
}

// Sixteen lanes hold 1024 elements of a row, a wave 4096, four waves 16384,
// sixteen 65536.  Short rows in number go to 16 lanes, rows that fit a wave to
// four where there are too few of them for every SIMD.
// Measured, us, rows x columns quantised (BF16), with the lanes: 65536 x 256 10 (16)
// and 25 (64), 16384 x 1024 7.4 and 10.2, 1024 x 1024 4.3 and 3.1; 16384 x 4096 31.3
// (64) and 33.9 (256), 1024 x 4096 4.7 and 4.4, 256 x 2048 3.5 and 3.1, 1 x 4096 4.0
// and 3.0; 8192 x 8192 50 (64), 30 (256) and 68 (1024), 8192 x 16384 62 (256) and 82
// (1024), 4096 x 32768 99 and 72.  The combined rows' gradient alike, choices x
// columns: 16384 x 512 8.2 (16) and 14.4 (64), 32 x 4096 5.4 (64) and 4.8 (256), 16384
// x 4096 52 and 64, 16384 x 8192 137 and 131 (but 8192 x 8192 52 and 60).
int row_lanes(int64_t rows, int64_t cols, int64_t cus) {
  if (cols > 16384) return 1024;
  if (cols <= 1024 && rows >= 32 * cus) return 16;
  return cols > 4096 || (cols > 512 && rows < 4 * cus) ? 256 : 64;
}

dense_gemm_status quantize_validate(int fmt, int64_t R, int64_t K, const void* X, int64_t ldx,
                                    int64_t x_rows, const void* rows, const void* Q, int64_t ldq,
                                    const void* S, bool* done) {
  *done = true;
  if (!valid_fmt(fmt)) return DENSE_GEMM_BAD_ARG;
  if (R < 0 || K < 0 || x_rows < 0) return DENSE_GEMM_INVALID_DIM;
  if (rows == nullptr && R > x_rows) return DENSE_GEMM_BAD_ARG;
  if (R == 0) return DENSE_GEMM_OK;
  if (R > kLayerMaxDim || K > kLayerMaxDim || x_rows > kLayerMaxDim) return DENSE_GEMM_TOO_LARGE;
  dense_gemm_status st = check_words(S, false);
  st = first_of(st, check_words(rows, true));
  if (K > 0) {
    if (x_rows > 0) st = first_of(st, check_rows(X, ldx, K));
    if (Q == nullptr) st = first_of(st, DENSE_GEMM_NULL_PTR);
    if (ldq < K) st = first_of(st, DENSE_GEMM_BAD_LD);
    if (ldq >= kMaxDim) st = first_of(st, DENSE_GEMM_TOO_LARGE);
  }
  *done = st != DENSE_GEMM_OK;
  return st;
}

static dense_gemm_status check_combine(int fmt, int64_t T, int64_t N, int64_t k, int64_t h_rows) {
  if (!valid_fmt(fmt)) return DENSE_GEMM_BAD_ARG;
  if (T < 0 || N < 0 || k < 0 || h_rows < 0) return DENSE_GEMM_INVALID_DIM;
  if (k == 0) return DENSE_GEMM_BAD_ARG;
  if (k > ROUTE_MOST_K || T > kLayerMaxDim / k || N > kLayerMaxDim || h_rows > kLayerMaxDim)
    return DENSE_GEMM_TOO_LARGE;
  return DENSE_GEMM_OK;
}

dense_gemm_status combine_validate(int fmt, int64_t T, int64_t N, int64_t k, const void* H, int64_t ldh,
                                   int64_t h_rows, const void* places, const void* weights,
                                   const void* residual, int64_t ldr, const void* Y, int64_t ldy,
                                   bool* done) {
  *done = true;
  dense_gemm_status st = check_combine(fmt, T, N, k, h_rows);
  if (st != DENSE_GEMM_OK || T == 0 || N == 0) return st;
  if (h_rows > 0) st = check_rows(H, ldh, N);
  st = first_of(st, check_words(places, false));
  st = first_of(st, check_words(weights, true));
  if (residual != nullptr) st = first_of(st, check_rows(residual, ldr, N));
  st = first_of(st, check_rows(Y, ldy, N));
  *done = st != DENSE_GEMM_OK;
  return st;
}

dense_gemm_status combine_grad_validate(int fmt, int64_t T, int64_t N, int64_t k, const void* DY,
                                        int64_t lddy, const void* H, int64_t ldh, int64_t h_rows,
                                        const void* places, const void* weights, const void* DH,
                                        int64_t lddh, const void* dweights, bool* done) {
  *done = true;
  dense_gemm_status st = check_combine(fmt, T, N, k, h_rows);
  if (st != DENSE_GEMM_OK || T == 0) return st;
  if (DH == nullptr && dweights == nullptr) return DENSE_GEMM_BAD_ARG;
  if (N == 0) return dweights != nullptr ? DENSE_GEMM_BAD_ARG : DENSE_GEMM_OK;
  st = check_rows(DY, lddy, N);
  if (dweights != nullptr && h_rows > 0) st = first_of(st, check_rows(H, ldh, N));
  st = first_of(st, check_words(places, false));
  st = first_of(st, check_words(weights, true));
  st = first_of(st, check_words(dweights, true));
  if (DH != nullptr) st = first_of(st, check_rows(DH, lddh, N));
  *done = st != DENSE_GEMM_OK;
  return st;
}

// ---- int8 products ----

namespace {

// Whether the LDS-DMA loads read a matrix of rows of K bytes in place: rows at
// 4-byte addresses, and for the tiled kernels (whose ranges end between words)
// of whole words.
bool direct_i8(const void* p, int64_t ld, int64_t stride, int64_t K, bool small) {
  return aligned(p, 4) && ((ld | stride) & 3) == 0 && (small || (K & 3) == 0);
}

int64_t round16(int64_t x) { return (x + 15) & ~(int64_t)15; }

bool copy_bytes(int64_t rows, int64_t K, size_t* out) {
  size_t n;
  if (__builtin_mul_overflow((size_t)rows, (size_t)round16(K), &n) || n > kMaxBytes - 256) return false;
  *out = (n + 255) & ~(size_t)255;
  return true;
}

const void* const kAligned = (const void*)(uintptr_t)256;

// Rows of pairs that stand for rows of K bytes in a plan.
int64_t pairs(int64_t K) { return 2 * ((K + 3) / 4); }

}  // namespace

dense_gemm_status i8_validate(int fmt, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* SA, const void* B, int64_t ldb, const void* SB,
                              const void* D, int64_t ldd, const dense_gemm_epilogue* e,
                              const dense_gemm_groups* g, int64_t sb_stride, bool* done) {
  *done = true;
  if (!valid_fmt(fmt)) return DENSE_GEMM_BAD_ARG;
  if (e != nullptr && e->grad != 0) return DENSE_GEMM_BAD_ARG;
  if (g != nullptr && sb_stride < 0) return DENSE_GEMM_BAD_ARG;
  if (K > I8_MOST_K) return DENSE_GEMM_TOO_LARGE;
  const bool some = M > 0 && N > 0 && (g == nullptr || g->count != 0);
  if (some && K > 0) {
    if (A == nullptr || B == nullptr) return DENSE_GEMM_NULL_PTR;
    if (lda < K || ldb < K) return DENSE_GEMM_BAD_LD;
    if (lda >= kMaxDim || ldb >= kMaxDim) return DENSE_GEMM_TOO_LARGE;
    // 32-bit offsets within a tile of rows, also of their copies
    const int64_t lim = ((int64_t)1 << 31) - 4096;
    if ((BM - 1) * (lda > ldb ? lda : ldb) + round16(K) >= lim) return DENSE_GEMM_TOO_LARGE;
  }
  // the rest are the checks of the 16-bit product
  const int64_t K2 = K < 0 ? K : pairs(K);
  const int64_t ld = K2 > 8 ? K2 : 8;
  const dense_gemm_status st = layer_validate(fmt == DENSE_GEMM_F16 ? DENSE_GEMM_NT_F16 : DENSE_GEMM_NT_BF16,
                                              M, N, K2, kAligned, ld, kAligned, ld, D, ldd, e, g, done);
  if (st != DENSE_GEMM_OK || *done) return st;
  const dense_gemm_status s = first_of(check_words(SA, false), check_words(SB, false));
  *done = s != DENSE_GEMM_OK;
  return s;
}

// The 16-bit plan as it stands.  Its estimate of a K step of 128 x 128 tiles over
// several rounds (79) is below what int8 takes, but where 110 would choose 256 x 256
// tiles instead the two are as fast, us, 128 against 256: 8192 x 8192 x 1024 91 and
// 97, x 1536 118 and 119, x 1664 124 and 123; 4096 x 4096 x 1024 25.1 and 25.2;
// 16384 x 4096 x 1024 91 and 91; 5000 x 5000 x 1500 67 and 66; 3000 x 5000 x 1024
// 26.1 and 25.6.
dense_gemm_status i8_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                          int64_t ldb, int64_t cus, CallPlan* cp) {
  const int64_t K2 = pairs(K);
  const dense_gemm_status st = layer_plan(NT, M, N, K2, kAligned, K2 + 8, kAligned, K2 + 8, cus, cp);
  if (st != DENSE_GEMM_OK) return st;
  cp->a_direct = K == 0 || direct_i8(A, lda, 0, K, cp->small());
  cp->b_direct = K == 0 || direct_i8(B, ldb, 0, K, cp->small());
  cp->a_bytes = cp->b_bytes = 0;
  if ((!cp->a_direct && !copy_bytes(M, K, &cp->a_bytes)) ||
      (!cp->b_direct && !copy_bytes(N, K, &cp->b_bytes)))
    return DENSE_GEMM_TOO_LARGE;
  return DENSE_GEMM_OK;
}

// With int8 values a K step holds twice the products for the same bytes, and 128
// x 128 tiles, which move twice the bytes of 256 x 256 ones per product, fall
// further behind than their 16-bit estimate (79) says: 110 decides as measured on
// all of these, us, 256 against 128: 16 groups of 256, N = K = 4096, 79 and 94; of
// 1024 235 and 331, K = 2048 144 and 197; 32 of 512, N = 2048, K = 4096, 130 and
// 167; 64 of 256, N = K = 2048, 87 and 107; 4 of 512, N = 512, K = 4096, 47 and 22;
// 48 of 300, N = 1400, K = 2000, 111 and 96; 128 of 200, N = 1024, K = 4096, 137
// and 191 (79 would take 128 there).
// The other two limits are the 16-bit products' as they stand.  Up to 192 rows a
// group on average 128 x 128 tiles: 16 groups of 128, N = K = 4096, 51 against 57
// in 256 x 256 tiles, 64 of 128, N = K = 2048, 57 and 72; past 128 rows int8 would
// be faster in those: 16 of 160, 75 and 58, 64 of 192, N = K = 2048, 89 and 77, 128
// of 160, N = 1024, K = 4096, 183 and 133.  The small-output kernel for few tiles:
// 8 groups of 1 to 16 rows, N = K = 4096, 34 to 37 against 35 in 128 x 128 tiles, 16
// of 4, N = K = 2048, 25 against 21; not taken: 32 groups, N = K = 2048, 45 to 48
// against 31.
dense_gemm_status i8_grouped_plan(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                  const void* B, int64_t ldb, const dense_gemm_groups& g, int64_t cus,
                                  GroupedPlan* out) {
  const int64_t K2 = pairs(K);
  dense_gemm_groups even = {g.ends, g.count, g.stride == 0 ? 0 : 8};
  const dense_gemm_status st = grouped_plan(NT, M, N, K2, kAligned, K2 + 8, kAligned, K2 + 8, even, cus, out,
                                            kNarrowStepI8);
  if (st != DENSE_GEMM_OK) return st;
  out->a_direct = K == 0 || direct_i8(A, lda, 0, K, out->small);
  out->b_direct = K == 0 || direct_i8(B, ldb, g.stride, K, out->small);
  out->a_bytes = out->b_bytes = 0;
  int64_t rows = 0;
  if ((!out->a_direct && !copy_bytes(M, K, &out->a_bytes)) ||
      (!out->b_direct && (__builtin_mul_overflow(out->matrices, N, &rows) ||
                          !copy_bytes(rows, K, &out->b_bytes))))
    return DENSE_GEMM_TOO_LARGE;
  return DENSE_GEMM_OK;
}

}  // namespace dg
