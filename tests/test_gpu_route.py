"""Routing to experts (dense_gemm_route, dense_gemm_route_grad) on the GPU,
against 64-bit plain forms: choices, ends, places and tokens equal, weights and
gradients within bounds derived in tests/_experts.py."""
import itertools
import math

import pytest

import dense_gemm_08_amd as dg
from dense_gemm_08_amd import binding
from tests import _experts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
S = binding.Status
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def logits(T, E, dtype, seed=0, sigma=1.5, ld=None):
    g = torch.Generator().manual_seed(1000 * T + E + seed)
    x = (torch.randn((T, E), generator=g) * sigma).to(TYPES[dtype])
    if ld is None:
        return x.cuda()
    wide = torch.full((max(T, 1), ld), math.nan, dtype=TYPES[dtype])  # (a read past a row shows)
    wide[:T, 1:1 + E] = x
    return wide.cuda()[:T, 1:1 + E]


def biases(E, seed=0, sigma=0.1):
    return (torch.randn(E, generator=torch.Generator().manual_seed(seed + E)) * sigma).cuda()


def run(l, k, what, **kw):
    print("route", tuple(l.shape), l.dtype, k, what, {a: b if not torch.is_tensor(b) else "bias" for a, b in kw.items()},
          flush=True)
    r = dg.route(l, k, **kw)
    torch.cuda.synchronize()
    _experts.check_route(r, l, k, what, **kw)
    return r


# every number of lanes and logits a lane, and both sides of each limit
EXPERTS = [1, 2, 5, 16, 17, 48, 64, 65, 127, 128, 129, 200, 256, 257, 300, 512, 513, 1000, 1024]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", EXPERTS)
def test_experts_and_choices(E, dtype):
    for T, k in ((1, 1), (3, min(E, 2)), (70, min(E, 8)), (130, min(E, 15)), (65, min(E, 16)), (5, min(E, 64))):
        l = logits(T, E, dtype)
        run(l, k, "softmax", renorm=True)
        run(l, k, "sigmoid biased", score="sigmoid", bias=biases(E), renorm=False, scale=2.5)
        run(l, k, "softmax biased", bias=biases(E, sigma=0.01), renorm=False)


@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 192, 1000, 4097, 33000])
def test_tokens(T):
    # (one block up to 128 tokens; blocks of 64; two chunks a block past 32768)
    for E, k, dtype in ((8, 2, "bf16"), (96, 6, "f32")):
        l = logits(T, E, dtype)
        r = run(l, k, "tokens", score="sigmoid", bias=biases(E))
        assert r.ends.shape == (E,) and int(r.ends[-1]) == T * k


@pytest.mark.parametrize("E,T", [(7, 40000), (130, 18001), (300, 9000), (513, 4160), (1024, 5000)])
def test_many_blocks(E, T):
    # (the blocks' counts in several passes of the placing launch, every row width;
    # two chunks a block past 32768 tokens)
    l = logits(T, E, "f16")
    l[::3, E // 2:] = -math.inf
    run(l, min(E, 5), "many blocks", score="sigmoid", bias=biases(E))


def test_many_tokens():
    l = logits(1 << 20, 4, "bf16")
    run(l, 1, "a million tokens")


GROUPS = [(16, 4, 2), (64, 8, 4), (256, 8, 4), (256, 8, 1), (256, 16, 7), (160, 5, 3), (96, 32, 9), (64, 64, 5),
          (63, 7, 2), (48, 2, 1), (512, 8, 3), (1024, 64, 33), (1000, 40, 11), (300, 3, 2), (128, 16, 16), (34, 17, 3)]


@pytest.mark.parametrize("E,groups,top", GROUPS)
def test_groups(E, groups, top):
    k = min(8, E // groups * top)
    for i, (dtype, score, biased, two) in enumerate(itertools.product(("f32", "bf16"), ("softmax", "sigmoid"),
                                                                      (False, True), (1, 2))):
        l = logits(75, E, dtype, seed=i)
        run(l, k, "groups", score=score, bias=biases(E, i) if biased else None, groups=groups, top_groups=top,
            group_top=two)


@pytest.mark.parametrize("E", [8, 64, 128, 256, 300, 700])
def test_ties_go_to_the_lowest_index(E):
    k = min(E, 8)
    for dtype in TYPES:
        l = logits(66, E, dtype, sigma=1.0)
        few = torch.round(l.float() * 2).to(l.dtype) / 2        # many equal logits
        same = torch.zeros_like(l)
        signs = torch.where(l > 0, 0.0, -0.0).to(l.dtype)       # both zeros
        for x, what in ((few, "few values"), (same, "all equal"), (signs, "zeros of both signs")):
            run(x, k, what)
            run(x, k, what + ", bias of zeros", score="sigmoid", bias=torch.zeros(E, device="cuda"))
            if E % 4 == 0:
                run(x, min(k, E // 2), what + ", groups", groups=4, top_groups=2, group_top=2, score="sigmoid")


@pytest.mark.parametrize("E", [16, 64, 200, 256, 513])
def test_scores_closer_than_32_bits_are_told_apart(E):
    # scores plus biases that differ by 2^-40 or so of their size: in 32 bits
    # these are equal, or the other way round
    k = min(8, E // 4)
    g = torch.Generator().manual_seed(E)
    for score in ("sigmoid", "softmax"):
        l = torch.randn((200, E), generator=g)
        s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), 1)
        bias = (0.75 - s[7]).float()  # token 7: all sums are 0.75 up to the bias's rounding
        r = run(l.cuda(), k, "near ties " + score, score=score, bias=bias.cuda(), renorm=False)
        c = (s[7] + bias.double())[r.experts[7].long().cpu()]
        assert float(c.max() - c.min()) < 2.0 ** -23 and float(c.max() - c.min()) > 0
        if E % 8 == 0:
            run(l.cuda(), k, "near ties of groups " + score, score=score, bias=bias.cuda(), groups=8,
                top_groups=4, group_top=2)
            run(l.cuda(), k, "sums of groups, no bias " + score, score=score, groups=8, top_groups=4, group_top=2)
        # many tokens whose choice has to be made again
        rows = l[7].repeat(150, 1)
        run(rows.cuda(), k, "all near ties " + score, score=score, bias=bias.cuda())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", [4, 48, 130, 256, 600])
def test_masked_experts_and_tokens(E, dtype):
    k = min(E, 6)
    l = logits(131, E, dtype)
    l[:, ::2] = -math.inf                   # half the experts are off
    l[5] = -math.inf                        # a token of padding
    l[6, 1:] = -math.inf                    # an expert that is off alone: none left
    l[7] = -math.inf
    l[7, 3] = 1.0                           # one left
    l[128:] = -math.inf                     # padding up to the end
    for kw in (dict(), dict(renorm=False), dict(score="sigmoid", bias=biases(E)), dict(bias=biases(E), renorm=False)):
        r = run(l, k, "masked", **kw)
        assert r.experts[5].tolist() == [-1] * k and r.weights[5].tolist() == [0.0] * k
        assert r.experts[7].tolist() == [3] + [-1] * (k - 1)
    n = int(r.ends[-1])
    assert (r.tokens[n:] == -1).all() and (r.tokens[:n] >= 0).all()
    if E % 4 == 0:
        for two in (1, 2):
            run(l, min(k, E // 4), "masked, groups", groups=4, top_groups=1, group_top=two, score="sigmoid")
    everything = torch.full((9, E), -math.inf, dtype=TYPES[dtype], device="cuda")
    assert run(everything, k, "nothing left").ends.tolist() == [0] * E
    # the type's lowest value is a number: such experts come last, with weight 0
    low = logits(10, E, dtype)
    low[:, 1:] = torch.finfo(TYPES[dtype]).min
    r = run(low, k, "lowest values")
    assert r.experts[0].tolist() == list(range(k)) and r.weights[0, 0] == 1.0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", [3, 64, 256, 520])
def test_broken_rows_are_routed_nowhere_and_show(E, dtype):
    l = logits(140, E, dtype)
    l[3, E - 1] = math.nan
    l[4, 0] = math.inf
    l[5] = math.nan
    l[6, 0] = -math.inf
    l[6, E - 1] = math.nan
    for kw in (dict(), dict(score="sigmoid", bias=biases(E)), dict(bias=biases(E), renorm=False)):
        r = run(l, min(E, 4), "broken rows", **kw)
        assert torch.isnan(r.weights[3:7]).all() and (r.experts[3:7] == -1).all()
        assert not torch.isnan(r.weights[:3]).any() and not torch.isnan(r.weights[7:]).any()


@pytest.mark.parametrize("E", [8, 64, 256, 300])
def test_biases_of_all_kinds(E):
    l = logits(100, E, "f32")
    for value in (-math.inf, math.inf, math.nan, -1e9, 1e9, -3.4e38):
        b = biases(E)
        b[1::3] = value
        run(l, min(4, E // 4), "bias %r" % value, score="sigmoid", bias=b)
        run(l, min(4, E // 4), "bias %r" % value, bias=b, groups=4, top_groups=2, group_top=2)
    run(l, 2, "no expert left", bias=torch.full((E,), -math.inf, device="cuda"))


def test_scores_that_underflow():
    # all chosen scores far below FP32's smallest: their weights still divide
    l = torch.full((3, 40), -math.inf, device="cuda")
    l[:, 4] = -500.0
    l[:, 9] = -500.5
    l[:, 30] = -700.0
    r = run(l, 3, "far below", score="sigmoid")
    assert abs(float(r.weights[0, 0]) - 1 / (1 + math.exp(-0.5))) < 1e-6
    l[:, 0] = 3.0
    run(l, 4, "beside a large one", score="sigmoid")
    run(l, 4, "beside a large one")


@pytest.mark.parametrize("E", [16, 64, 256, 512, 1024])
def test_masks_of_the_lowest_value(E):
    # in the logits these can still be chosen, in the bias too, where the sums of
    # two for a group pass FP32's range
    k, low = 6, torch.finfo(torch.float32).min
    for dtype in TYPES:
        l = logits(90, E, dtype)
        l[:, ::3] = torch.finfo(TYPES[dtype]).min
        l[4] = torch.finfo(TYPES[dtype]).min
        for kw in (dict(), dict(renorm=False), dict(score="sigmoid", bias=biases(E)),
                   dict(score="sigmoid", groups=4, top_groups=2, group_top=2)):
            run(l, k, "lowest logits", **kw)
        l = logits(90, E, dtype, seed=1)
        for off in (E // 4 - 1, E // 2, 3 * E // 4 + 1, E):  # (one group stays, two, none whole)
            bias = biases(E)
            bias[E - off:] = low
            for groups in (4, 8) if E < 512 else (4, 32):
                for top in (2, groups - 1):
                    if E // groups * top >= k:
                        r = run(l, k, "lowest biases", score="sigmoid", bias=bias, groups=groups, top_groups=top,
                                group_top=2)
                        assert int(r.ends[-1]) == 90 * k
        bias[:E // 4] = 0.5 * low
        bias[E // 4:E // 2] = 0.75 * low
        run(l, k, "low biases", bias=bias, groups=4, top_groups=2, group_top=2)


def test_strides():
    for dtype in TYPES:
        for E, ld in ((48, 51), (256, 300), (130, 133)):
            l = logits(70, E, dtype, ld=ld)
            assert l.stride(0) == ld
            run(l, 4, "strided", score="sigmoid", bias=biases(E))
            _grad(l, 4, "softmax", False, 1.0)


def _grad(l, k, score, renorm, scale, missing=False):
    T, E = l.shape
    r = dg.route(l, k, score=score, renorm=renorm, scale=scale)
    e = r.experts.clone()
    if missing:
        e[::3, k - 1] = -1
        e[1::5] = -1
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(T + E)).cuda()
    print("route_grad", tuple(l.shape), l.dtype, k, score, renorm, scale, missing, flush=True)
    d = dg.route_grad(l, e, dw, score=score, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    _experts.check_route_grad(d, l, e, dw, score, renorm, scale, "route_grad")
    return d


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", [1, 2, 16, 17, 48, 64, 65, 128, 200, 256, 257, 512, 777, 1024])
def test_gradient(E, dtype):
    for T, k in ((1, 1), (17, min(E, 6)), (100, min(E, 17)), (3, min(E, 64))):
        for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
            l = logits(T, E, dtype)
            _grad(l, k, score, renorm, 2.5)
            _grad(l, k, score, renorm, 1.0, missing=True)


def test_gradient_of_masked_rows_is_zero_there():
    l = logits(40, 64, "f32")
    l[:, 10:20] = -math.inf
    l[7] = -math.inf
    for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
        d = _grad(l, 4, score, renorm, 1.0)
        assert (d[:, 10:20] == 0).all() and (d[7] == 0).all()


@pytest.mark.parametrize("score,renorm", list(itertools.product(("softmax", "sigmoid"), (True, False))))
def test_gradient_against_differences(score, renorm):
    # 64-bit central differences of the weights at the choice made: their error is
    # h^2 / 6 times a third derivative (below 8 here) plus 2^-52 / h: under 1e-8
    l = logits(6, 40, "f32", sigma=1.0)
    r = dg.route(l, 5, score=score, renorm=renorm, scale=1.5)
    dw = torch.randn((6, 5), generator=torch.Generator().manual_seed(3)).cuda()
    d = dg.route_grad(l, r.experts, dw, score=score, renorm=renorm, scale=1.5).cpu().double()
    x, e, h = l.cpu().double(), r.experts.cpu().long(), 1e-5
    for i in range(40):
        up, down = x.clone(), x.clone()
        up[:, i] += h
        down[:, i] -= h
        f = [(_experts.weights64(y, e, score, renorm, 1.5) * dw.cpu().double()).sum(1) for y in (up, down)]
        # (the library's own error: relative 2^-20 of the terms, which are below 8)
        assert float(((f[0] - f[1]) / (2 * h) - d[:, i]).abs().max()) < 1e-7 + 8 * 2.0 ** -20


def test_choices_outside_the_experts_take_no_part():
    l = logits(20, 30, "bf16")
    e = torch.randint(0, 30, (20, 3), dtype=torch.int32, device="cuda")
    for bad in (-1, -2147483648, 30, 2147483647):
        e[::2, 1] = bad
        dw = torch.randn((20, 3), device="cuda")
        for score, renorm in itertools.product(("softmax", "sigmoid"), (True, False)):
            d = dg.route_grad(l, e, dw, score=score, renorm=renorm)
            _experts.check_route_grad(d, l, e, dw, score, renorm, 1.0, "outside %d" % bad)


def test_results_repeat():
    l = logits(5000, 256, "bf16")
    kw = dict(score="sigmoid", bias=biases(256), groups=8, top_groups=4, group_top=2)
    a = dg.route(l, 8, **kw)
    for _ in range(3):
        b = dg.route(l, 8, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_python_refusals():
    l = logits(8, 16, "f32")
    e = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((8, 2), device="cuda")
    for call in (lambda: dg.route(l[0], 2), lambda: dg.route(l.t(), 2), lambda: dg.route(l, 2, score="max"),
                 lambda: dg.route(l, 2, bias=torch.zeros(15, device="cuda")), lambda: dg.route(l, -1),
                 lambda: dg.route(l, 2, bias=torch.zeros(16)), lambda: dg.route_grad(l, e[:7], w),
                 lambda: dg.route_grad(l, e, w[:, :1]), lambda: dg.route_grad(l, e, w, D=l[:, :15]),
                 lambda: dg.route_grad(l, e.t(), w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dg.route(l.double(), 2), lambda: dg.route(l, 2, bias=torch.zeros(16, device="cuda").half()),
                 lambda: dg.route_grad(l, e.long(), w), lambda: dg.route_grad(l, e, w.half())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: dg.route(l, 0), lambda: dg.route(l, 17), lambda: dg.route(l, 2, groups=3),
                 lambda: dg.route(l, 9, groups=2, top_groups=1)):
        with pytest.raises(dg.DenseGemmError) as err:
            call()
        assert err.value.status == S.BAD_ARG
    with pytest.raises(dg.DenseGemmError) as err:
        dg.route(l, 1 << 40)
    assert err.value.status == S.TOO_LARGE
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(dg.DenseGemmError) as err:
        dg.route(logits(200, 16, "f32"), 2, workspace=small)
    assert err.value.status == S.WORKSPACE_TOO_SMALL
