"""The int8 products (dense_gemm_i8) on the GPU, against products that are exact
in 64-bit floats; bounds of the scales, the epilogue and the rounding as derived
in tests/_experts.py."""
import itertools
import math

import pytest

import dense_gemm_08_amd as dg
from dense_gemm_08_amd import binding
from tests import _experts, _i8_cases, _layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
S = binding.Status
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = list(binding.ACTS)


def gen(*key):
    seed = 17
    for k in key:
        seed = (seed * 1000003 + k) % (1 << 31)
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(shape, g, at=0, ld=None):
    """int8 values of the whole range, -128 among them; with ld a view into rows
    of ld bytes that begin `at` bytes on, other values around it."""
    if ld is None:
        return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    rows = math.prod(shape[:-1])
    flat = torch.randint(-128, 128, (rows * ld + at + 16,), generator=g, device="cuda", dtype=torch.int8)
    strides = [1]
    for n in reversed((ld,) + tuple(shape[1:-1])[::-1]):
        strides.insert(0, strides[0] * n if len(strides) > 1 else n)
    if len(shape) == 2:
        return flat[at:].as_strided(shape, (ld, 1))
    return flat[at:].as_strided(shape, (shape[1] * ld, ld, 1))


def operands(M, N, K, dtype, g, G=(), **kw):
    dt = TYPES[dtype]
    A, B = codes((M, K), g, **kw), codes(G + (N, K), g, **kw)
    SA = torch.rand(M, generator=g, device="cuda") * 0.02 + 0.001
    SB = (torch.rand(G + (N,), generator=g, device="cuda") * 0.02 + 0.001) / max(K, 1) ** 0.5
    bias = torch.randn(G + (N,), generator=g, device="cuda").to(dt)
    res = torch.randn((M, N), generator=g, device="cuda").to(dt)
    return A, SA, B, SB, bias, res


def run(M, N, K, dtype, bias, act, residual, keep, what="", **kw):
    print("gemm_nt_i8", M, N, K, dtype, bias, act, residual, keep, kw, what, flush=True)
    A, SA, B, SB, b, r = operands(M, N, K, dtype, gen(M, N, K), **kw)
    Z = torch.full((M, N), 9.0, dtype=TYPES[dtype], device="cuda") if keep else None
    D = dg.gemm_nt_i8(A, SA, B, SB, bias=b if bias else None, act=act, residual=r if residual else None,
                      preact=Z, dtype=TYPES[dtype])
    torch.cuda.synchronize()
    _experts.check_i8(D, Z, A, SA, B, SB, b if bias else None, act, r if residual else None, what)
    return D


@pytest.mark.parametrize("case", _i8_cases.I8, ids=str)
def test_every_kernel(case):
    i = _i8_cases.I8.index(case)
    run(*case, list(TYPES)[i % 2], i % 3 != 0, ACTS[i % 5], i % 2 == 1, i % 4 == 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K", [0, 1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 131, 255, 257, 1000, 1023])
def test_lengths_of_the_sum(K, dtype):
    for M, N in ((1, 1), (5, 70), (16, 16), (40, 33), (129, 130), (300, 257)):
        run(M, N, K, dtype, True, "silu", True, True)


@pytest.mark.parametrize("M,N", [(1, 4096), (16, 17), (17, 16), (128, 128), (129, 128), (128, 129), (255, 257),
                                 (256, 256), (513, 100), (100, 513), (1, 2), (2, 1), (640, 1)])
def test_outputs(M, N):
    for K, dtype in ((260, "f16"), (1024, "bf16")):
        for act, residual, keep in itertools.product(ACTS, (False, True), (False, True)):
            run(M, N, K, dtype, keep != residual, act, residual, keep)


@pytest.mark.parametrize("at,more", [(0, 0), (1, 0), (2, 0), (3, 1), (4, 4), (0, 1), (0, 2), (0, 3), (5, 8), (8, 24)])
def test_operands_anywhere(at, more):
    # read in place or copied, small-output kernel and tiled ones; the bytes around
    # the rows are not zeros
    for M, N, K in ((9, 100, 77), (9, 100, 128), (70, 90, 515), (200, 260, 77), (200, 260, 132), (300, 129, 2048)):
        run(M, N, K, "bf16", True, "none", False, False, at=at, ld=K + more)


def test_largest_sums():
    # -128 everywhere: the largest K gives 2^31 - 16384, one short of overflow
    for M, N in ((3, 5), (130, 140), (300, 300)):
        K = 131071
        A = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        B = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
        B[1] = 127
        one = torch.ones(max(M, N), device="cuda")
        D = dg.gemm_nt_i8(A, one[:M] / 65536, B, one[:N] / 1024)
        want = torch.full((M, N), 128 * 128 * K / 2.0 ** 26, dtype=torch.float64, device="cuda")
        want[:, 1] *= -127 / 128
        _layer.assert_close(D, want, want.abs() * (2.0 ** -8 + 4 * _layer.U), "largest sums")
    with pytest.raises(dg.DenseGemmError) as e:
        A = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
        dg.gemm_nt_i8(A, one[:1], A, one[:1])
    assert e.value.status == S.TOO_LARGE


def test_scales_of_all_sizes():
    A, SA, B, SB, bias, res = operands(70, 300, 400, "bf16", gen(3))
    for sa, sb in ((1e-30, 1e30), (1e30, 1e-30), (0.0, 1.0), (1e-20, 1e-10), (2.0 ** 60, 2.0 ** 60)):
        x, y = SA * sa, SB * sb
        _experts.check_i8(dg.gemm_nt_i8(A, x, B, y), None, A, x, B, y, None, "none", None, "scales")
    x = SA.clone()
    x[3], x[4] = math.nan, math.inf
    D = dg.gemm_nt_i8(A, x, B, SB)
    assert torch.isnan(D[3]).all() and not torch.isfinite(D[4]).any()
    rest = [i for i in range(70) if i not in (3, 4)]
    _experts.check_i8(D[rest], None, A[rest], SA[rest], B, SB, None, "none", None, "others")


def test_residual_in_place_and_strided_outputs():
    for M, N, K in ((9, 100, 260), (300, 300, 512), (300, 264, 9000)):
        A, SA, B, SB, bias, res = operands(M, N, K, "f16", gen(M, N))
        want = dg.gemm_nt_i8(A, SA, B, SB, bias=bias, act="gelu", residual=res)
        same = res.clone()
        assert dg.gemm_nt_i8(A, SA, B, SB, bias=bias, act="gelu", residual=same, D=same) is same
        assert torch.equal(same, want)
        wide = torch.full((M, N + 13), 7.0, dtype=torch.float16, device="cuda")
        zw = torch.full((M, N + 5), 8.0, dtype=torch.float16, device="cuda")
        rw = torch.full((M, N + 3), 9.0, dtype=torch.float16, device="cuda")
        rw[:, 1:1 + N] = res
        dg.gemm_nt_i8(A, SA, B, SB, bias=bias, act="gelu", residual=rw[:, 1:1 + N], preact=zw[:, 3:3 + N],
                      D=wide[:, 5:5 + N])
        assert torch.equal(wide[:, 5:5 + N], want)
        wide[:, 5:5 + N] = 7.0
        zw[:, 3:3 + N] = 8.0
        assert (wide == 7.0).all() and (zw == 8.0).all()


def test_the_plan_changes_nothing():
    # the sums are exact: a row of a large product, of a split one and of a small
    # one are the same bits
    K, N = 9000, 300
    A, SA, B, SB, bias, res = operands(700, N, K, "bf16", gen(5))
    whole = dg.gemm_nt_i8(A, SA, B, SB, bias=bias, act="silu")
    for lo, hi in ((0, 1), (3, 20), (100, 228), (0, 300), (650, 700)):
        assert torch.equal(dg.gemm_nt_i8(A[lo:hi], SA[lo:hi], B, SB, bias=bias, act="silu"), whole[lo:hi])
    ends = torch.tensor([100, 700], dtype=torch.int32, device="cuda")
    two = dg.gemm_nt_i8_grouped(A, SA, torch.stack([B, B]), torch.stack([SB, SB]), ends,
                                bias=torch.stack([bias, bias]), act="silu")
    assert torch.equal(two, whole)


def spread(rows, G, g):
    cut = torch.sort(torch.randint(0, rows + 1, (G - 1,), generator=g, device="cuda")).values
    return torch.cat([cut, torch.full((1,), rows, device="cuda")]).to(torch.int32)


def check_grouped(M, N, K, G, dtype, ends, act="silu", shared=False, tail=0, **kw):
    g = gen(M, N, K, G)
    A, SA, B, SB, bias, res = operands(M + tail, N, K, dtype, g, G=(1 if shared else G,), **kw)
    if shared:
        B, SB, bias = [x.expand((G,) + x.shape[1:]) for x in (B, SB, bias)]
        SB = SB.contiguous()
    SA[M:] = math.nan
    D = torch.full((M + tail, N), 7.0, dtype=TYPES[dtype], device="cuda")
    Z = torch.full_like(D, 8.0)
    res[M:] = math.nan
    print("grouped", M, N, K, G, dtype, act, shared, tail, kw, flush=True)
    dg.gemm_nt_i8_grouped(A, SA, B, SB, ends, bias=bias, act=act, residual=res, preact=Z, D=D)
    torch.cuda.synchronize()
    last = 0
    for i, end in enumerate(ends.tolist()):
        # (an end below the one before it counts as that one)
        lo, hi = last, min(max(end, last), M + tail)
        last = hi
        if lo < hi:
            _experts.check_i8(D[lo:hi], Z[lo:hi], A[lo:hi], SA[lo:hi], B[i], SB[i], bias[i], act, res[lo:hi],
                              "group %d" % i)
    assert (D[last:] == 7.0).all() and (Z[last:] == 8.0).all()


@pytest.mark.parametrize("case", _i8_cases.GROUPED, ids=str)
def test_every_grouped_kernel(case):
    rows, N, K, G = case
    i = _i8_cases.GROUPED.index(case)
    check_grouped(rows, N, K, G, list(TYPES)[i % 2], spread(rows, G, gen(i)), act=ACTS[i % 5])
    check_grouped(rows, N, K, G, list(TYPES)[1 - i % 2], spread(rows, G, gen(i + 99)), act="none", tail=37)


def test_groups_of_all_shapes():
    for ends in ([0, 0, 0], [0, 40, 40], [40, 40, 40], [1, 2, 40], [16, 32, 33], [0, 0, 40], [7, 7, 30]):
        e = torch.tensor(ends, dtype=torch.int32, device="cuda")
        for N, K in ((70, 100), (300, 515)):
            check_grouped(40, N, K, 3, "f16", e, tail=5)
    e = torch.tensor([300, 300, 900, 901], dtype=torch.int32, device="cuda")
    check_grouped(1000, 300, 260, 4, "bf16", e, tail=11)
    check_grouped(1000, 300, 260, 4, "bf16", e, shared=True)
    check_grouped(1000, 300, 262, 4, "bf16", e, at=3, ld=263)
    check_grouped(1000, 300, 261, 4, "bf16", e, shared=True)


def test_ends_that_lead_outside_stay_inside():
    for ends in ([-5, 20, 99], [30, 10, 40], [2147483647, 0, -2147483648]):
        check_grouped(40, 90, 128, 3, "bf16", torch.tensor(ends, dtype=torch.int32, device="cuda"))


def test_no_groups():
    A, SA, B, SB, bias, res = operands(5, 6, 8, "bf16", gen(1))
    D = torch.full((5, 6), 77.0, dtype=torch.bfloat16, device="cuda")
    dg.gemm_nt_i8_grouped(A, SA, B.new_empty((0, 6, 8)), SB.new_empty((0, 6)),
                          torch.empty(0, dtype=torch.int32, device="cuda"), D=D)
    assert (D == 77.0).all()
    assert dg.gemm_nt_i8(A[:0], SA[:0], B, SB).shape == (0, 6)
    assert dg.gemm_nt_i8(A, SA, B[:0], SB[:0]).shape == (5, 0)


def test_workspaces():
    A, SA, B, SB, bias, res = operands(300, 300, 9001, "bf16", gen(2))
    want = dg.gemm_nt_i8(A, SA, B, SB)
    with pytest.raises(dg.DenseGemmError) as e:
        dg.gemm_nt_i8(A, SA, B, SB, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.status == S.WORKSPACE_TOO_SMALL
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(dg.gemm_nt_i8(A, SA, B, SB, workspace=ws), want)
    with pytest.raises(dg.DenseGemmError) as e:
        dg.gemm_nt_i8(A, SA, B, SB, workspace=ws[16:])
    assert e.value.status == S.MISALIGNED


def test_python_refusals():
    A, SA, B, SB, bias, res = operands(6, 10, 16, "bf16", gen(7))
    ends = torch.tensor([6], dtype=torch.int32, device="cuda")
    for call in (lambda: dg.gemm_nt_i8(A[0], SA, B, SB), lambda: dg.gemm_nt_i8(A.t(), SA, B, SB),
                 lambda: dg.gemm_nt_i8(A, SA[:5], B, SB), lambda: dg.gemm_nt_i8(A, SA, B, SB[:9]),
                 lambda: dg.gemm_nt_i8(A, SA, B[:, :8], SB), lambda: dg.gemm_nt_i8(A, SA.cpu(), B, SB),
                 lambda: dg.gemm_nt_i8(A, SA, B, torch.ones(20, device="cuda")[::2]),
                 lambda: dg.gemm_nt_i8(A, SA, B, SB, act="tanh"), lambda: dg.gemm_nt_i8(A, SA, B, SB, bias=bias[:9]),
                 lambda: dg.gemm_nt_i8(A, SA, B, SB, residual=res[:5]), lambda: dg.gemm_nt_i8(A, SA, B, SB, D=res.t()),
                 lambda: dg.gemm_nt_i8_grouped(A, SA, B, SB, ends), lambda: dg.gemm_nt_i8_grouped(A, SA, B[None], SB, ends),
                 lambda: dg.gemm_nt_i8_grouped(A, SA, B[None], SB[None], ends.repeat(2))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dg.gemm_nt_i8(A.float(), SA, B, SB), lambda: dg.gemm_nt_i8(A, SA, B.view(torch.uint8), SB),
                 lambda: dg.gemm_nt_i8(A, SA.half(), B, SB), lambda: dg.gemm_nt_i8(A, SA, B, SB, dtype=torch.float32),
                 lambda: dg.gemm_nt_i8(A, SA, B, SB, bias=bias.half(), residual=res),
                 lambda: dg.gemm_nt_i8(A, SA, B, SB, bias=bias.half(), D=res),
                 lambda: dg.gemm_nt_i8_grouped(A, SA, B[None], SB[None], ends.long())):
        with pytest.raises(TypeError):
            call()
