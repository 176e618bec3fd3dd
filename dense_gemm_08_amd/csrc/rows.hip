// rows.hip -- rows around an expert layer's products (dense_gemm_quantize_i8,
// dense_gemm_combine and its gradient, include/dense_gemm.h) on the MI355X
// (gfx950).  Host side; the kernels are in rows_kernel.h.
#include "layer_host.h"
#include "plan_experts.h"
#include "rows_kernel.h"

namespace dg {

namespace {

// f(W) for rows shared by W lanes.
template <typename Launch>
void by_lanes(int lanes, Launch&& launch) {
  if (lanes == 16)
    launch(std::integral_constant<int, 16>());
  else if (lanes == 64)
    launch(std::integral_constant<int, 64>());
  else if (lanes == 256)
    launch(std::integral_constant<int, 256>());
  else
    launch(std::integral_constant<int, 1024>());
}

// Workgroups for so many rows; fewer than 2^32 threads.
unsigned row_grid(int64_t rows, int64_t per) {
  const int64_t blocks = (rows + per - 1) / per, most = 1 << 21;
  return (unsigned)(blocks < most ? blocks : most);
}

template <typename T>
dense_gemm_status run_quantize(const QuantizeParams& p, int lanes, hipStream_t stream) {
  by_lanes(lanes, [&](auto w) {
    constexpr int W = decltype(w)::value;
    hipLaunchKernelGGL((quantize_rows_i8<T, W>), dim3(row_grid(p.count, rows_per_block<W>())),
                       dim3(row_threads<W>()), 0, stream, p);
  });
  return launched();
}

template <typename T>
dense_gemm_status run_combine_grad(const CombineGradParams& p, int lanes, hipStream_t stream) {
  by_lanes(lanes, [&](auto w) {
    constexpr int W = decltype(w)::value;
    hipLaunchKernelGGL((combine_rows_grad<T, W>), dim3(row_grid(p.count * p.k, rows_per_block<W>())),
                       dim3(row_threads<W>()), 0, stream, p);
  });
  return launched();
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

dense_gemm_status dense_gemm_quantize_i8(int fmt, int64_t R, int64_t K, const void* X, int64_t ldx,
                                         int64_t x_rows, const void* rows, void* Q, int64_t ldq, void* S,
                                         hipStream_t stream) {
  bool done;
  dense_gemm_status st = quantize_validate(fmt, R, K, X, ldx, x_rows, rows, Q, ldq, S, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  int cus, xcds;
  st = device_topology(&cus, &xcds);
  if (st != DENSE_GEMM_OK) return st;
  const QuantizeParams p = {(const uint16_t*)X, (const int32_t*)rows, (int8_t*)Q, (float*)S,
                            ldx, ldq, R, x_rows, (int)K};
  const int lanes = row_lanes(R, K, cus);
  return fmt == DENSE_GEMM_BF16 ? run_quantize<__bf16>(p, lanes, stream)
                                : run_quantize<_Float16>(p, lanes, stream);
}

dense_gemm_status dense_gemm_combine(int fmt, int64_t T, int64_t N, int64_t k, const void* H, int64_t ldh,
                                     int64_t h_rows, const void* places, const void* weights,
                                     const void* residual, int64_t ldr, void* Y, int64_t ldy,
                                     hipStream_t stream) {
  bool done;
  dense_gemm_status st = combine_validate(fmt, T, N, k, H, ldh, h_rows, places, weights, residual, ldr, Y,
                                          ldy, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  int cus, xcds;
  st = device_topology(&cus, &xcds);
  if (st != DENSE_GEMM_OK) return st;
  CombineParams p = {(const uint16_t*)H, (const int32_t*)places, (const float*)weights,
                     (const uint16_t*)residual, (uint16_t*)Y, ldh, ldr, ldy, T, h_rows, (int)N, (int)k, 1};
  while (p.lanes < 256 && p.lanes * 8 < N) p.lanes *= 2;
  const int64_t pieces = (N + p.lanes * 8 - 1) / (p.lanes * 8);
  // (fewer than 2^32 threads, and fewer than 2^16 rows of workgroups)
  const unsigned x = row_grid(T, 256 / p.lanes);
  int64_t y = ((int64_t)1 << 23) / x;
  if (y > 65535) y = 65535;
  const dim3 grid(x, (unsigned)(pieces < y ? pieces : y));
  if (fmt == DENSE_GEMM_BF16)
    hipLaunchKernelGGL(combine_rows<__bf16>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(combine_rows<_Float16>, grid, dim3(256), 0, stream, p);
  return launched();
}

dense_gemm_status dense_gemm_combine_grad(int fmt, int64_t T, int64_t N, int64_t k, const void* DY,
                                          int64_t lddy, const void* H, int64_t ldh, int64_t h_rows,
                                          const void* places, const void* weights, void* DH, int64_t lddh,
                                          void* dweights, hipStream_t stream) {
  bool done;
  dense_gemm_status st = combine_grad_validate(fmt, T, N, k, DY, lddy, H, ldh, h_rows, places, weights, DH,
                                               lddh, dweights, &done);
  if (st != DENSE_GEMM_OK || done) return st;
  int cus, xcds;
  st = device_topology(&cus, &xcds);
  if (st != DENSE_GEMM_OK) return st;
  const CombineGradParams p = {(const uint16_t*)DY, (const uint16_t*)H, (const int32_t*)places,
                               (const float*)weights, (uint16_t*)DH, (float*)dweights, lddy, ldh, lddh, T,
                               h_rows, (int)N, (int)k};
  const int lanes = row_lanes(T * k, N, cus);
  return fmt == DENSE_GEMM_BF16 ? run_combine_grad<__bf16>(p, lanes, stream)
                                : run_combine_grad<_Float16>(p, lanes, stream);
}

}  // extern "C"
