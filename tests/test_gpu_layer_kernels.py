"""Every kernel of the layer products on the GPU (tests/_layer_cases.py lists
calls that launch each of them on 256 CUs), output by output.

* Small integers, with ReLU: every product, bias, residual and FP32 partial sum
  is a whole number below 2^24, so whatever the order of the sums each output is
  the correctly rounded exact value.  A dropped, doubled or misplaced row, tile,
  part or column sum shows.
* Normal values with an activation that is not exact, against 64-bit forms
  within the bounds of tests/_layer.py."""
import numpy as np
import pytest
import torch

import dense_gemm_08_amd as dg
from tests import _layer as L
from tests import _layer_cases as cases

pytestmark = pytest.mark.gpu

LAYOUTS = ("nt", "nn")
FUSED = (dg.gemm_nt_fused, dg.gemm_nn_fused)
DACT = (dg.gemm_nt_dact, dg.gemm_nn_dact)
GROUPED = (dg.gemm_nt_grouped, dg.gemm_nn_grouped)
GROUPED_DACT = (dg.gemm_nt_grouped_dact, dg.gemm_nn_grouped_dact)
CANARY = 77.0
both = pytest.mark.parametrize("dtype", ["f16", "bf16"])


def generator(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) % (1 << 31))


def ints(gen, *shape, dt, top=3):
    assert 9 * 40000 + 2 * top < 2 ** 24
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(dt)


def normals(gen, *shape, dt, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dt)


def product(A, B, layout):
    """A.B^ of small integers, exactly (in 64 bits)."""
    b = B.double()
    return A.double() @ (b.t().contiguous() if layout == 0 else b)


def exactly(got, want, what):
    want = want.to(got.dtype)
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError("%s: %d of %d differ, first at %s: %r, not %r" % (
            what, bad.shape[0], got.numel(), i, got[i].item(), want[i].item()))


def uneven(rows, groups):
    """Row counts: some groups empty, one with near half of the rows, the last
    not empty."""
    rng = np.random.default_rng(rows * 31 + groups)
    share = rng.exponential(size=groups) ** 2 * (rng.random(groups) < 0.8)
    share[rng.integers(groups)] = max(share.sum(), 1.0)
    sizes = rng.multinomial(rows, share / share.sum())
    if sizes[-1] == 0:
        sizes[int(sizes.argmax())] -= 1
        sizes[-1] = 1
    return [int(s) for s in sizes]


def spans(sizes):
    ends = np.cumsum(sizes).tolist()
    return list(zip([0] + ends[:-1], ends)), torch.tensor(ends, dtype=torch.int32, device="cuda")


@both
@pytest.mark.parametrize("layout,M,N,K", cases.LAYER)
def test_layer(layout, M, N, K, dtype):
    dt = L.GEN[dtype]
    gen = generator(M, N, K)
    shape = (N, K) if layout == 0 else (K, N)
    A, B, bias, res = (ints(gen, *s, dt=dt) for s in ((M, K), shape, (N,), (M, N)))
    P = product(A, B, layout)
    Z = torch.empty((M, N), dtype=dt, device="cuda")
    D = FUSED[layout](A, B, bias=bias, act="relu", residual=res, preact=Z)
    exactly(Z, P + bias.double(), "Z")
    exactly(D, (P + bias.double()).clamp(min=0) + res.double(), "D")
    exactly(DACT[layout](A, B, res, "relu"), P * (res > 0), "gradient")
    del P, Z, D
    A, B = normals(gen, M, K, dt=dt), normals(gen, *shape, dt=dt, sigma=K ** -0.5)
    D = FUSED[layout](A, B, bias=bias, act="silu")
    L.check_forward(D, None, A, B, LAYOUTS[layout], bias, "silu", None, "silu")


@both
@pytest.mark.parametrize("layout,M,N,K,G", cases.GROUPED)
def test_grouped(layout, M, N, K, G, dtype):
    dt = L.GEN[dtype]
    gen = generator(M, N, K, G)
    groups, ends = spans(uneven(M, G))
    pad = 5
    A, B = ints(gen, M + pad, K, dt=dt), ints(gen, *((G, N, K) if layout == 0 else (G, K, N)), dt=dt)
    bias, res = ints(gen, G, N, dt=dt), ints(gen, M + pad, N, dt=dt)
    A[M:] = float("nan")  # rows of no group
    D, Z, dZ = (torch.full((M + pad, N), CANARY, dtype=dt, device="cuda") for _ in range(3))
    GROUPED[layout](A, B, ends, bias=bias, act="relu", residual=res, preact=Z, D=D)
    GROUPED_DACT[layout](A, B, ends, res, "relu", D=dZ)
    for g, (lo, hi) in enumerate(groups):
        if hi > lo:
            P = product(A[lo:hi], B[g], layout)
            exactly(Z[lo:hi], P + bias[g].double(), "Z %d" % g)
            exactly(D[lo:hi], (P + bias[g].double()).clamp(min=0) + res[lo:hi].double(), "D %d" % g)
            exactly(dZ[lo:hi], P * (res[lo:hi] > 0), "gradient %d" % g)
    for t in (D, Z, dZ):
        assert bool((t[M:] == CANARY).all())


@both
@pytest.mark.parametrize("M,N,K,G,sums", cases.TN)
def test_tn(M, N, K, G, sums, dtype):
    dt = L.GEN[dtype]
    gen = generator(M, N, K, G)
    A, B = ints(gen, K, M, dt=dt), ints(gen, K, N, dt=dt)
    if G == 0:
        got = dg.gemm_tn(A, B, colsum=bool(sums))
        D, c = got if sums else (got, None)
        exactly(D, A.double().t().contiguous() @ B.double(), "D")
        if sums:
            exactly(c, A.double().sum(0), "sums")
        return
    groups, ends = spans(uneven(K, G))
    got = dg.gemm_tn_grouped(A, B, ends, colsum=bool(sums))
    D, c = got if sums else (got, None)
    for g, (lo, hi) in enumerate(groups):
        a = A[lo:hi].double()
        exactly(D[g], a.t().contiguous() @ B[lo:hi].double(), "D %d" % g)
        if sums:
            exactly(c[g], a.sum(0), "sums %d" % g)
