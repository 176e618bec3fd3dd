"""Rows of D wider than one workgroup per 16 columns allows: a launch holds
fewer than 2^32 threads (past that the runtime reports no error, and the
products were left almost wholly uncomputed), the small-output kernels take 512
for each 16 columns."""
import ctypes

import pytest

from dense_gemm_08_amd import binding

S = binding.Status
WIDEST = (2 ** 32 - 1) // 512 * 16  # columns in the small-output kernels' tiles


def test_plans_of_wide_rows():
    lib = binding.load_library()
    out = (ctypes.c_int64 * 16)()
    for M in (1, 16):
        for K in (0, 8):
            for layout in (0, 1):
                for N in (WIDEST - 5, WIDEST, WIDEST + 1, 2 ** 31 - 1024):
                    assert lib.dense_gemm_plan(layout, M, N, K, 256, out) == S.OK
                    if out[7] == 512:
                        assert out[3] * out[4] * 512 < 2 ** 32, (layout, M, N, K)
                    if layout == 0:
                        assert (out[7] == 512) == (N <= WIDEST), (M, N, K)
        for N in (WIDEST, WIDEST + 1):
            assert lib.gemm_nt_e4m3_mx_plan(M, N, 64, 256, out) == S.OK
            assert (out[7] == 512) == (N <= WIDEST)


@pytest.mark.gpu
def test_products_of_wide_rows():
    import torch
    import dense_gemm_08_amd as dg
    N = WIDEST + 17
    col = torch.arange(N, device="cuda") % 7
    A = torch.ones((2, 8), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((N, 8), dtype=torch.bfloat16, device="cuda")
    B[:, 3] = col
    none = torch.empty((0, N), dtype=A.dtype, device="cuda")
    rows = torch.stack([B[:, 3]] * 2)
    for f in (lambda: dg.gemm_nt_bf16(A, B), lambda: dg.gemm_nt_fused(A, B, act="relu"),
              lambda: dg.gemm_nn_fused(A[:, :0], none, residual=rows)):
        D = f()
        torch.cuda.synchronize()
        right = bool((D == col).all())
        assert right and D.shape == (2, N)
    del B
    one = torch.full((2, 1), 127, dtype=torch.uint8, device="cuda")
    A8 = torch.full((2, 32), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    B8 = torch.zeros((N, 32), dtype=torch.uint8, device="cuda")
    B8[:, 5] = torch.where(col > 3, 0x38, 0).to(torch.uint8)
    D = dg.gemm_nt_e4m3_mx(A8, one, B8, torch.full((N, 1), 127, dtype=torch.uint8, device="cuda"))
    right = bool((D == (col > 3)).all())
    assert right
