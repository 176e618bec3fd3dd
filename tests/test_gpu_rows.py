"""Rows quantised to int8 and the experts' rows combined (dense_gemm_quantize_i8,
dense_gemm_combine and its gradient) on the GPU, against 64-bit plain forms:
whole numbers and scales equal, sums within bounds derived in
tests/_experts.py."""
import math

import pytest

import dense_gemm_08_amd as dg
from tests import _experts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def values(R, K, dtype, seed=0, ld=None, at=0):
    g = torch.Generator().manual_seed(100003 * R + K + seed)
    x = (torch.randn((R, K), generator=g) * torch.exp(torch.randn((R, 1), generator=g))).to(TYPES[dtype])
    if ld is None:
        return x.cuda()
    wide = torch.full((R, ld), math.nan, dtype=TYPES[dtype])  # (a read past a row shows)
    wide[:, at:at + K] = x
    return wide.cuda()[:, at:at + K]


def check(x, Q, S, what):
    q, s = _experts.quantized(x)
    assert torch.equal(S.cpu().nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0)), (what, "scales")
    if not torch.equal(Q.cpu(), q):
        i = tuple(torch.nonzero(Q.cpu() != q)[0].tolist())
        raise AssertionError("%s: %d differ, first at %r: %d, want %d of %r" % (
            what, int((Q.cpu() != q).sum()), i, Q[i], q[i], x[i].item()))


def run(x, what):
    print("quantize_rows", tuple(x.shape), x.dtype, x.stride(), what, flush=True)
    Q, S = dg.quantize_rows(x)
    torch.cuda.synchronize()
    check(x, Q, S, what)


# both sides of what 16 lanes, a wave, four and sixteen hold, and more than that
COLUMNS = [1, 2, 7, 8, 9, 63, 127, 128, 129, 511, 512, 513, 1000, 1023, 1024, 1025, 4095, 4096, 4097, 16383,
           16384, 16385, 65535, 65536, 65537, 140001]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K", COLUMNS)
def test_quantize_columns(K, dtype):
    run(values(1, K, dtype), "one row")
    run(values(5, K, dtype), "rows")
    run(values(3, K, dtype, ld=K + 5, at=3), "odd rows")


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 15, 16, 17, 63, 1023, 1024, 8191, 8192, 8193, 20000])
def test_quantize_rows(R):
    for K in (24, 200, 1024, 1025):
        run(values(R, K, "bf16"), "rows")


def test_quantize_nothing():
    for dtype in TYPES.values():
        Q, S = dg.quantize_rows(torch.empty((0, 40), dtype=dtype, device="cuda"))
        assert Q.shape == (0, 40) and S.shape == (0,)
        Q, S = dg.quantize_rows(torch.empty((7, 0), dtype=dtype, device="cuda"))
        assert Q.shape == (7, 0) and S.tolist() == [0.0] * 7


def test_quantize_every_value():
    # all finite FP16 and BF16 values, in rows whose largest value is each power of
    # two times something odd: half-way cases, subnormals, the largest numbers
    for dtype in TYPES.values():
        bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
        all_values = bits.view(dtype)
        finite = all_values[torch.isfinite(all_values.float())]
        mags = finite.float().abs()
        tops = torch.unique(mags[mags > 0])
        tops = tops[torch.linspace(0, len(tops) - 1, 400).long()]
        rows = []
        for t in tops.tolist():
            inside = finite[mags <= t]
            pick = torch.randperm(len(inside), generator=torch.Generator().manual_seed(int(t * 7) % 99991))[:1500]
            row = torch.zeros(1501, dtype=dtype)
            row[:len(pick)] = inside[pick]
            row[1500] = t
            rows.append(row)
        run(torch.stack(rows).cuda(), "every value")


def test_quantize_half_way_cases():
    # m = 254 a: x = (2 i + 1) a lies half-way between i and i + 1; m = 127 a: x = i a
    # is whole, x = (i + 1/2) a half-way
    for dtype in TYPES.values():
        for a in (1.0, 0.25, 2.0 ** -9, 2.0 ** 5):
            x = torch.zeros((2, 300))
            x[0, :127] = (2 * torch.arange(127) + 1) * a
            x[0, 127:254] = -(2 * torch.arange(127) + 1) * a
            x[0, 299] = 254 * a
            x[1, :127] = torch.arange(127) * a
            x[1, 127:253] = (torch.arange(126) + 0.5) * a
            x[1, 299] = -127 * a
            t = x.to(dtype)
            assert torch.equal(t.float()[0], x[0])
            run(t.cuda(), "half-way")
            Q, _ = dg.quantize_rows(t.cuda())
            want = torch.round((2 * torch.arange(127) + 1) / 2.0).to(torch.int8)
            assert torch.equal(Q[0, :127].cpu(), want) and torch.equal(Q[0, 127:254].cpu(), -want)


@pytest.mark.parametrize("K", [5, 64, 1500, 5000, 20000])
def test_quantize_special_rows(K):
    for dtype in TYPES:
        x = values(12, K, dtype)
        x[1] = 0.0
        x[2] = -0.0
        x[3, K - 1] = math.inf
        x[4, 0] = -math.inf
        x[5, K // 2] = math.nan
        x[6] = torch.finfo(x.dtype).max
        x[7] = torch.finfo(x.dtype).min
        x[8] = torch.finfo(x.dtype).smallest_normal / 2     # subnormal throughout
        x[9] = x[9] * torch.finfo(x.dtype).smallest_normal
        x[10] = torch.finfo(x.dtype).tiny
        x[10, 1] = torch.finfo(x.dtype).max
        run(x, "special rows")
        Q, S = dg.quantize_rows(x)
        assert torch.isnan(S[3:6]).all() and (Q[1:6] == 0).all() and (S[1:3] == 0).all()


def test_quantize_gathered():
    for dtype in TYPES:
        for K in (40, 1000, 4100):
            x = values(50, K, dtype)
            rows = torch.randint(0, 50, (133,), dtype=torch.int32)
            rows[[3, 60, 132]] = torch.tensor([-1, 50, 2147483647], dtype=torch.int32)
            rows[4] = -2147483648
            print("gathered", K, dtype, flush=True)
            Q, S = dg.quantize_rows(x, rows=rows.cuda())
            inside = (rows >= 0) & (rows < 50)
            src = torch.where(inside[:, None], x.cpu()[rows.long().clamp(0, 49)], torch.zeros((), dtype=x.dtype))
            check(src, Q, S, "gathered")
    # no row of X at all
    Q, S = dg.quantize_rows(torch.empty((0, 24), dtype=torch.float16, device="cuda"),
                            rows=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert (Q == 0).all() and (S == 0).all()


def test_quantize_into_given_outputs():
    x = values(33, 77, "bf16")
    for ldq, at in ((80, 0), (81, 1), (79, 2), (90, 7)):
        wide = torch.full((33, ldq), 99, dtype=torch.int8, device="cuda")
        Q = wide[:, at:at + 77]
        S = torch.empty(33, device="cuda")
        got = dg.quantize_rows(x, Q=Q, S=S)
        assert got[0] is Q and got[1] is S
        check(x, Q, S, "given")
        wide[:, at:at + 77] = 99
        assert (wide == 99).all()  # nothing beside the columns was written


def test_more_rows_than_a_launch_has_workgroups():
    # 2^21 workgroups of 16 rows, and some more rows in turn
    R, K = (1 << 25) + 1000, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((R, K), generator=g, device="cuda", dtype=torch.float16)
    print("quantize_rows", R, K, flush=True)
    Q, S = dg.quantize_rows(x)
    for lo in range(0, R, 1 << 23):
        part = x[lo:lo + (1 << 23)].double()
        m = part.abs().amax(1, keepdim=True)
        assert torch.equal(Q[lo:lo + (1 << 23)], torch.round(part * 127 / m).to(torch.int8))
        assert torch.equal(S[lo:lo + (1 << 23)], (m[:, 0] / 127).float())


def test_very_long_rows():
    # more pieces of a row than a grid has rows of workgroups; segments of a row
    N = 65535 * 2048 + 5003
    h = (torch.arange(N, device="cuda") % 1021).to(torch.float16).view(1, N)
    p = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    w = torch.full((1, 1), 2.0, device="cuda")
    print("combine", N, flush=True)
    assert torch.equal(dg.combine_rows(h, p, w), 2 * h)
    dh, dw = dg.combine_rows_grad(h, h, p, w)
    assert torch.equal(dh, 2 * h)
    total = float((h.double() ** 2).sum())
    # (a lane's sum of N / 1024 products, and the lanes')
    assert abs(float(dw) - total) <= (N / 1024 + 16) * 2.0 ** -24 * total
    Q, S = dg.quantize_rows(h)
    assert float(S) == torch.tensor(1020 / 127, dtype=torch.float64).float().item()
    assert torch.equal(Q[0], torch.round((torch.arange(N, device="cuda") % 1021).double() * 127 / 1020).to(torch.int8))


def choices(T, k, R, seed=0, missing=0.0):
    g = torch.Generator().manual_seed(T * 31 + k + seed)
    p = torch.randperm(max(R, T * k), generator=g)[:T * k].view(T, k).to(torch.int32)
    p = torch.where(torch.rand((T, k), generator=g) < missing, torch.full_like(p, -1), p)
    w = torch.rand((T, k), generator=g) + 0.05
    return p.cuda(), (w / w.sum(1, keepdim=True)).cuda()


COMBINE = [(1, 1, 1), (1, 8, 2), (3, 7, 1), (5, 16, 3), (64, 9, 2), (33, 129, 5), (7, 1000, 4), (130, 1024, 8),
           (17, 1025, 6), (9, 4096, 2), (4, 4097, 3), (3, 16384, 2), (2, 16400, 9), (2, 70001, 2), (2000, 64, 2),
           (9000, 40, 3), (3000, 1001, 4), (11, 24, 64), (6, 2056, 33)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,N,k", COMBINE)
def test_combine_and_gradient(T, N, k, dtype):
    R = T * k + 3
    h = values(R, N, dtype, seed=1)
    for missing in (0.0, 0.3):
        p, w = choices(T, k, R, missing=missing)
        res = values(T, N, dtype, seed=2)
        print("combine", T, N, k, dtype, missing, flush=True)
        for ww, rr in ((w, None), (None, None), (w, res), (None, res)):
            _experts.check_combine(dg.combine_rows(h, p, ww, residual=rr), h, p, ww, rr, "combine")
        dy = values(T, N, dtype, seed=3)
        for ww in (w, None):
            before = torch.full((R, N), 3.0, dtype=TYPES[dtype], device="cuda")
            dh, dw = dg.combine_rows_grad(dy, h, p, ww, dh=before.clone())
            _experts.check_combine_grad(dh, dw, dy, h, p, ww, before, "combine_grad")


def test_combine_strides_and_places_outside():
    for dtype in TYPES:
        h = values(40, 77, dtype, ld=83, at=3)
        p, w = choices(13, 3, 40)
        p[2, 1], p[3, 0], p[4, 2], p[5, 1] = 40, -1, 2147483647, -2147483648
        res = values(13, 77, dtype, seed=5, ld=79, at=1)
        wide = torch.full((13, 90), 5.0, dtype=TYPES[dtype], device="cuda")
        y = wide[:, 5:82]
        assert dg.combine_rows(h, p, w, residual=res, D=y) is y
        _experts.check_combine(y, h, p, w, res, "strided")
        same = res.clone()
        dg.combine_rows(h, p, w, residual=same, D=same)     # in place
        assert torch.equal(same, y)
        y.fill_(5.0)
        assert (wide == 5.0).all()
        dy = values(13, 77, dtype, seed=6, ld=91, at=7)
        hwide = torch.full((40, 99), 6.0, dtype=TYPES[dtype], device="cuda")
        before = hwide[:, 9:86].clone()
        dh, dw = dg.combine_rows_grad(dy, h, p, w, dh=hwide[:, 9:86])
        _experts.check_combine_grad(dh, dw, dy, h, p, w, before, "strided")
        assert dw[2, 1] == 0 and dw[3, 0] == 0
        hwide[:, 9:86] = 6.0
        assert (hwide == 6.0).all()


def test_combine_the_same_row_twice():
    h = values(5, 130, "bf16")
    p = torch.tensor([[1, 1], [1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.25, 0.5], [1.0, 2.0]], device="cuda")
    _experts.check_combine(dg.combine_rows(h, p, w), h, p, w, None, "twice")
    dy = values(2, 130, "bf16", seed=2)
    dh, dw = dg.combine_rows_grad(dy, h, p, w)
    both = [(w[t, j] * dy[t].float()).bfloat16() for t, j in ((0, 0), (0, 1), (1, 0))]
    picked = torch.stack([dh[1] == b for b in both]).any(0)
    assert picked.all() and torch.equal(dh[0], (2 * dy[1].float()).bfloat16())


def test_weights_that_are_nan_show():
    h = values(4, 40, "f16")
    p = torch.tensor([[0, -1], [-1, -1], [2, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, math.nan], [math.nan, math.nan], [1.0, 1.0]], device="cuda")
    y = dg.combine_rows(h, p, w)
    assert torch.isnan(y[:2]).all() and not torch.isnan(y[2]).any()


def test_no_rows():
    h = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    res = values(3, 24, "bf16")
    assert torch.equal(dg.combine_rows(h, p, w, residual=res), res)
    dh, dw = dg.combine_rows_grad(res, h, p, w)
    assert dh.shape == (0, 24) and (dw == 0).all()
    assert dg.combine_rows(res, p[:0], w[:0]).shape == (0, 24)
    assert dg.combine_rows(res[:, :0], p, w).shape == (3, 0)


def test_combine_gradient_against_differences():
    # the combination is linear in h and in the weights: 64-bit differences of the
    # plain form are exact up to rounding, the library's gradients to a step of
    # their type
    h, (p, w) = values(12, 9, "f16"), choices(4, 3, 12)
    dy = values(4, 9, "f16", seed=1)
    dh, dw = dg.combine_rows_grad(dy, h, p, w, dh=torch.zeros_like(h))

    def loss(hh, ww):
        r, _ = _experts.rows64(hh, p)
        return ((r * ww[:, :, None]).sum(1) * dy.double()).sum()

    for i, j in ((0, 0), (5, 3), (11, 8), (7, 2)):
        up, down = h.double().clone(), h.double().clone()
        up[i, j] += 0.5
        down[i, j] -= 0.5
        d = float(loss(up, w.double()) - loss(down, w.double()))
        assert abs(d - float(dh[i, j])) <= 2.0 ** -11 * abs(d) + 2.0 ** -24
    for t, j in ((0, 0), (3, 2), (1, 1)):
        up, down = w.double().clone(), w.double().clone()
        up[t, j] += 0.5
        down[t, j] -= 0.5
        d = float(loss(h.double(), up) - loss(h.double(), down))
        S = float((dy.double()[t] * h.double()[p[t, j].long()]).abs().sum())
        assert abs(d - float(dw[t, j])) <= 25 * 2.0 ** -24 * S + 1e-12


def test_python_refusals():
    x = values(6, 16, "bf16")
    i = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((6, 2), device="cuda")
    for call in (lambda: dg.quantize_rows(x[0]), lambda: dg.quantize_rows(x.t()), lambda: dg.quantize_rows(x, rows=i),
                 lambda: dg.quantize_rows(x, rows=i[:, 0]), lambda: dg.quantize_rows(x, rows=i[:, 0].cpu()),
                 lambda: dg.quantize_rows(x, S=w), lambda: dg.quantize_rows(x, Q=torch.empty((6, 15), dtype=torch.int8, device="cuda")),
                 lambda: dg.combine_rows(x, i[0]), lambda: dg.combine_rows(x, i.t()), lambda: dg.combine_rows(x, i, w[:, :1]),
                 lambda: dg.combine_rows(x, i, w, residual=x[:5]), lambda: dg.combine_rows(x, i, w, D=x[:, :8]),
                 lambda: dg.combine_rows_grad(x[:5], x, i, w), lambda: dg.combine_rows_grad(x, x, i, w, dh=x[:5]),
                 lambda: dg.combine_rows(x, i.cpu(), w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dg.quantize_rows(x.float()), lambda: dg.quantize_rows(x, rows=i[:, 0].contiguous().long()),
                 lambda: dg.combine_rows(x, i.long()), lambda: dg.combine_rows(x, i, w.half()),
                 lambda: dg.combine_rows(x, i, w, residual=x.half()), lambda: dg.combine_rows_grad(x.half(), x, i, w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(dg.DenseGemmError):
        dg.combine_rows_grad(x[:, :0], x[:, :0], i, w)  # dweights of nothing
