"""Masked loads at the largest operand spans the argument checks accept.

The kernels mask a lane's load by giving it the buffer offset OOB
(csrc/cdna_ops.h), which has to lie past every range.  The first K step's
range begins koff elements before the tile's rows (so that the last step ends
at K), so it is up to a K step longer than the span the argument checks bound
by 2^31 bytes.  Were OOB inside it, the places before k = 0 would hold values
of the tile's last row in place of zeros.
"""
import ctypes
import os
import re

import pytest

from dense_gemm_08_amd import binding

S = binding.Status
HERE = os.path.dirname(os.path.abspath(__file__))
ROWS = 256  # a tile's
NT_F16 = dict(M=512, N=512, ld=4210008, K=189768)
MX = dict(M=256, N=256, ld=8400064, K=5467296)


def oob():
    src = open(os.path.join(os.path.dirname(HERE), "dense_gemm_08_amd", "csrc", "cdna_ops.h")).read()
    return int(re.search(r"constexpr uint32_t OOB = (0x[0-9a-f]+)u;", src).group(1), 16)


def range16(ld, K, whole):
    """Bytes of the first K step's range of a 16-bit operand whose rows of K
    values are rounded up to `whole` elements."""
    Kw = (K + whole - 1) // whole * whole
    return 2 * ((ROWS - 1) * ld + Kw + -Kw % 64)


def accepted16(ld, K):
    p = ctypes.c_void_p(256)
    return binding.load_library().dense_gemm_validate(0, 512, 512, K, p, ld, p, ld, p, 512) == S.OK


def test_masking_offset_lies_past_every_accepted_range():
    far = oob()
    assert far < 2 ** 32 - (1 << 20)  # (an offset may be added to it)
    worst = 0
    for ld in range(4194304, 4210752, 2):
        most = (2 ** 30 - 9 - (ROWS - 1) * ld) // 8 * 8  # the largest K that fits, a multiple of 8
        if not 0 < most <= ld:
            continue
        for K in range(most, max(most - 64, 0), -2):
            for whole in (2, 8):
                worst = max(worst, range16(ld, K, whole))
    # (the sizes of the regression below are accepted and reach that far)
    assert accepted16(NT_F16["ld"], NT_F16["K"])
    assert 2 ** 31 < range16(NT_F16["ld"], NT_F16["K"], 8) <= worst
    assert worst <= far


def mx_range(ld, K):
    return (ROWS - 1) * ld + K + -K % 128


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="made-up pointers")
def test_masking_offset_lies_past_the_block_scaled_products_ranges():
    fn = binding.raw("gemm_nt_e4m3_mx")
    ld, K = MX["ld"], MX["K"]
    assert S(fn(256, 256, K, 256, ld, 256, K // 32, 256, ld, 256, K // 32, 256, 256, None)) == S.NO_DEVICE
    assert 2 ** 31 < mx_range(ld, K) <= oob()


def zeros(rows, ld, dtype):
    import torch
    return torch.zeros((rows, ld), dtype=dtype, device="cuda")


@pytest.mark.gpu
def test_nt_values_of_the_last_row_stay_out_of_the_sums():
    import torch
    import dense_gemm_08_amd as dg
    n, ld, K = ROWS, NT_F16["ld"], NT_F16["K"]
    at = 2 ** 30 - (-K % 64) - (n - 1) * ld  # the last row's column at buffer offset 2^31
    assert 0 < at < K
    print("A.B^T %d x %d x %d, lda = ldb = %d" % (n, n, K, ld), flush=True)
    A, B = zeros(n, ld, torch.float16), zeros(n, ld, torch.float16)
    A[n - 1, at:at + 8] = 1.0
    B[n - 1, at:at + 8] = 1.0
    want = torch.zeros((n, n), dtype=torch.float16, device="cuda")
    want[n - 1, n - 1] = 8.0
    assert torch.equal(dg.gemm_nt_f16(A[:, :K], B[:, :K]), want)
    assert torch.equal(dg.gemm_nt_fused(A[:, :K], B[:, :K]), want)


@pytest.mark.gpu
def test_layer_infinities_of_the_last_row_stay_there():
    import torch
    import dense_gemm_08_amd as dg
    # 256-row tiles (more 128 x 128 tiles than a round, over 16 K steps), rows
    # of K values that are not whole 16-byte pieces
    n, N = ROWS, 33024
    for K in range(1090, 1 << 17, 64):
        ld = (2 ** 30 - 9 - (K + 6)) // (n - 1) // 2 * 2
        if range16(ld, K, 2) >= 2 ** 31 + 16:
            break
    at = 2 ** 30 - 62 - (n - 1) * ld
    assert accepted16(ld, K) and K % 64 == 2 and 0 < at < K
    print("layer A.B %d x %d x %d, lda = %d" % (n, N, K, ld), flush=True)
    A = zeros(n, ld, torch.bfloat16)
    A[n - 1, at:K] = float("inf")
    B = torch.ones((K, N), dtype=torch.bfloat16, device="cuda")
    D = dg.gemm_nn_fused(A[:, :K], B)
    assert bool((D[:n - 1] == 0).all())
    assert bool((D[n - 1] == float("inf")).all())


@pytest.mark.gpu
def test_block_scaled_values_of_the_last_row_stay_out_of_the_sums():
    import torch
    import dense_gemm_08_amd as dg
    n, ld, K = ROWS, MX["ld"], MX["K"]
    at = 2 ** 31 - (-K % 128) - (n - 1) * ld
    assert 0 < at < K
    print("FP8 block-scaled A.B^T %d x %d x %d, lda = ldb = %d" % (n, n, K, ld), flush=True)
    A, B = zeros(n, ld, torch.uint8), zeros(n, ld, torch.uint8)
    A[n - 1, at:at + 16] = 0x38  # 1.0
    B[n - 1, at:at + 16] = 0x38
    one = torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")  # 2^0
    want = torch.zeros((n, n), dtype=torch.bfloat16, device="cuda")
    want[n - 1, n - 1] = 16.0
    assert torch.equal(dg.gemm_nt_e4m3_mx(A[:, :K], one, B[:, :K], one), want)
