"""MI355X (gfx950) tiled dense GEMM: D = A.B^T (FP16) and D = A.B (BF16), the
FP8 block-scaled D = A.B^T (E4M3 with E8M0 scales per 32 K values), and the
products of a transformer's dense and expert layers: bias, activation and
residual in the epilogue, the input, weight and bias gradients, and a weight
matrix per group of rows; the same products in int8 with a scale per row of each
operand; and what stands around an expert layer's products: routing, rows
quantised, rows combined.

The arithmetic runs in the hand-written HIP kernels of ``libdense_gemm.so``
(built from ``csrc/``).  This package only marshals arguments to its C ABI;
importing it does not load the library, and every call fails loudly if the
library is missing.
"""
from .binding import (  # noqa: F401
    Status,
    DenseGemmError,
    gemm_nt_f16,
    gemm_nn_bf16,
    gemm_nt_bf16,
    gemm_nn_f16,
    gemm_nt_e4m3_mx,
    gemm_nt_fused,
    gemm_nn_fused,
    gemm_nt_dact,
    gemm_nn_dact,
    gemm_tn,
    gemm_nt_grouped,
    gemm_nn_grouped,
    gemm_nt_grouped_dact,
    gemm_nn_grouped_dact,
    gemm_tn_grouped,
    gemm_nt_i8,
    gemm_nt_i8_grouped,
    quantize_rows,
    Routes,
    route,
    route_grad,
    combine_rows,
    combine_rows_grad,
    library_path,
    load_library,
)
