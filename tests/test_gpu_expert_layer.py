"""Whole expert layers on the GPU: routing, the experts' products and their rows
brought back, served in int8 and trained in 16 bits, each stage checked against its
64-bit form from the values that the stage before it left; the same in captured
graphs, on another stream, by two threads and with a padded batch."""
import math
import threading

import pytest

import dense_gemm_08_amd as dg
from tests import _experts, _layer

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Layer:
    """An expert layer: E experts of two products, F features inside."""

    def __init__(self, E, N, F, dtype, seed=0, **routing):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.router = torch.randn((E, N), generator=g, device="cuda").to(dtype) / N ** 0.5
        self.w1 = (torch.randn((E, F, N), generator=g, device="cuda") / N ** 0.5).to(dtype)
        self.w2 = (torch.randn((E, N, F), generator=g, device="cuda") / F ** 0.5).to(dtype)
        self.b1 = (torch.randn((E, F), generator=g, device="cuda") * 0.3).to(dtype)
        self.k, self.E, self.F, self.N = routing.pop("k"), E, F, N
        self.routing = routing
        self.q1, self.s1 = [x.view(E, F, -1).squeeze(-1) if x.dim() == 1 else x.view(E, F, N)
                            for x in dg.quantize_rows(self.w1.view(E * F, N))]
        self.q2, self.s2 = [x.view(E, N, -1).squeeze(-1) if x.dim() == 1 else x.view(E, N, F)
                            for x in dg.quantize_rows(self.w2.view(E * N, F))]

    def logits(self, x):
        return dg.gemm_nt_fused(x, self.router)

    def serve(self, x, logits=None, stream=None):
        l = self.logits(x) if logits is None else logits
        r = dg.route(l, self.k, stream=stream, **self.routing)
        q, s = dg.quantize_rows(x, rows=r.tokens, stream=stream)
        h = dg.gemm_nt_i8_grouped(q, s, self.q1, self.s1, r.ends, bias=self.b1, act="silu", dtype=x.dtype,
                                  stream=stream)
        q2, s2 = dg.quantize_rows(h, stream=stream)
        y = dg.gemm_nt_i8_grouped(q2, s2, self.q2, self.s2, r.ends, dtype=x.dtype, stream=stream)
        return dict(l=l, r=r, q=q, s=s, h=h, q2=q2, s2=s2, y=y,
                    out=dg.combine_rows(y, r.places, r.weights, residual=x, stream=stream))

    def check(self, x, v):
        r = v["r"]
        _experts.check_route(r, v["l"], self.k, "route", **self.routing)
        n = int(r.ends[-1])
        at = r.tokens[:n].long()
        q, s = _experts.quantized(x[at])
        assert torch.equal(v["q"][:n].cpu(), q) and torch.equal(v["s"][:n].cpu(), s)
        assert (v["q"][n:] == 0).all() and (v["s"][n:] == 0).all()
        q, s = _experts.quantized(v["h"][:n])
        assert torch.equal(v["q2"][:n].cpu(), q) and torch.equal(v["s2"][:n].cpu(), s)
        for e, lo, hi in _layer.spans(r.ends.tolist()):
            if lo < hi:
                _experts.check_i8(v["h"][lo:hi], None, v["q"][lo:hi], v["s"][lo:hi], self.q1[e], self.s1[e],
                                  self.b1[e], "silu", None, "first")
                _experts.check_i8(v["y"][lo:hi], None, v["q2"][lo:hi], v["s2"][lo:hi], self.q2[e], self.s2[e],
                                  None, "none", None, "second")
        _experts.check_combine(v["out"], v["y"], r.places, r.weights, x, "out")


def tokens(T, N, dtype, seed=1):
    return torch.randn((T, N), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


CONFIGS = [
    (16, 200, 136, torch.bfloat16, dict(k=2)),
    (64, 256, 320, torch.bfloat16, dict(k=6, score="sigmoid", groups=8, top_groups=3, group_top=2, scale=2.5)),
    (5, 77, 101, torch.float16, dict(k=3, renorm=False)),
]


@pytest.mark.parametrize("config", CONFIGS, ids=["16", "64-groups", "odd"])
@pytest.mark.parametrize("T", [1, 3, 16, 130, 700])
def test_served_in_int8(config, T):
    E, N, F, dtype, kw = config
    layer = Layer(E, N, F, dtype, **kw)
    x = tokens(T, N, dtype)
    v = layer.serve(x)
    torch.cuda.synchronize()
    layer.check(x, v)
    # the whole of it near the layer in 64 bits: int8 rounding, 1 / 254 of a row's
    # largest value in each operand of two products, leaves a few percent
    r, xd = v["r"], x.double()
    y = xd.clone()
    for t in range(T):
        for j in range(layer.k):
            e = int(r.experts[t, j])
            h = torch.nn.functional.silu(layer.w1[e].double() @ xd[t] + layer.b1[e].double())
            y[t] += float(r.weights[t, j]) * (layer.w2[e].double() @ h)
        if t >= 20:
            y, got = y[:t + 1], v["out"][:t + 1]
            break
    else:
        got = v["out"]
    inner = (y - xd[:len(y)]).norm()
    assert float((got.double() - y).norm()) < 0.1 * float(inner) + 2.0 ** -8 * float(y.norm())


def test_a_padded_batch():
    E, N, F, dtype, kw = CONFIGS[1]
    layer = Layer(E, N, F, dtype, bias=torch.zeros(64, device="cuda"), **kw)
    x = tokens(40, N, dtype)
    full = layer.serve(x[:29].contiguous())
    x[29:] = math.nan                       # what the padding holds changes nothing
    l = torch.full((40, E), -math.inf, dtype=dtype, device="cuda")
    l[:29] = full["l"]
    v = layer.serve(x, logits=l)
    assert torch.equal(v["out"][:29], full["out"])
    assert torch.isnan(v["out"][29:]).all()  # (its own rows pass through by the skip connection)
    assert int(v["r"].ends[-1]) == 29 * layer.k and (v["r"].tokens[29 * layer.k:] == -1).all()


def test_on_another_stream():
    E, N, F, dtype, kw = CONFIGS[0]
    layer = Layer(E, N, F, dtype, **kw)
    x = tokens(300, N, dtype)
    want = layer.serve(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer.serve(x, logits=want["l"], stream=s)
    raw = layer.serve(x, logits=want["l"], stream=s.cuda_stream)
    s.synchronize()
    for name in ("q", "h", "q2", "y", "out"):
        n = int(want["r"].ends[-1])
        assert torch.equal(got[name][:n], want[name][:n]) and torch.equal(raw[name][:n], want[name][:n])


def test_two_threads():
    E, N, F, dtype, kw = CONFIGS[1]
    layer = Layer(E, N, F, dtype, **kw)
    xs = [tokens(200, N, dtype, seed=s) for s in (1, 2)]
    want = [layer.serve(x)["out"] for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                if not torch.equal(layer.serve(xs[i])["out"], want[i]):
                    wrong.append(i)
        torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("T", [4, 16, 300])
def test_captured_graphs(T):
    # two graphs over one layer, replayed in turn with eager work in between and new
    # inputs each time
    E, N, F, dtype, kw = CONFIGS[1]
    layer = Layer(E, N, F, dtype, **kw)
    ins = [tokens(T, N, dtype, seed=s) for s in (1, 2)]
    for x in ins:
        layer.serve(x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for x in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(layer.serve(x))
        graphs.append(g)
    for rep in range(4):
        for i in (0, 1):
            ins[i].copy_(tokens(T, N, dtype, seed=10 * rep + i))
        for i in (0, 1, 0):
            graphs[i].replay()
            torch.cuda.synchronize()
            want = layer.serve(ins[i])
            n = int(want["r"].ends[-1])
            for name in ("q", "h", "y", "out"):
                rows = slice(0, n) if name != "out" else slice(None)
                assert torch.equal(outs[i][name][rows], want[name][rows]), (rep, i, name)
            for a, b in zip(outs[i]["r"], want["r"]):
                assert torch.equal(a, b)
    layer.check(ins[0], outs[0])


@pytest.mark.parametrize("config", [CONFIGS[0], CONFIGS[2],
                                    (32, 128, 96, torch.bfloat16, dict(k=4, score="sigmoid"))],
                         ids=["16", "odd", "sigmoid"])
def test_trained_in_16_bits(config):
    # forward and backward, each stage from the values that the library's own one
    # before it left
    E, N, F, dtype, kw = config
    layer = Layer(E, N, F, dtype, **kw)
    T = 150
    x, dout = tokens(T, N, dtype), tokens(T, N, dtype, seed=9)
    l = layer.logits(x)
    r = dg.route(l, layer.k, **layer.routing)
    _experts.check_route(r, l, layer.k, "route", **layer.routing)
    xs = x[r.tokens.long()]
    z = torch.empty((T * layer.k, F), dtype=dtype, device="cuda")
    h = dg.gemm_nt_grouped(xs, layer.w1, r.ends, bias=layer.b1, act="silu", preact=z)
    y = dg.gemm_nt_grouped(h, layer.w2, r.ends)
    out = dg.combine_rows(y, r.places, r.weights, residual=x)
    _experts.check_combine(out, y, r.places, r.weights, x, "out")
    before = torch.zeros_like(y)
    dy, dw = dg.combine_rows_grad(dout, y, r.places, r.weights, dh=before.clone())
    _experts.check_combine_grad(dy, dw, dout, y, r.places, r.weights, before, "combine_grad")
    dz = dg.gemm_nn_grouped_dact(dy, layer.w2, r.ends, z, "silu")
    dxs = dg.gemm_nn_grouped(dz, layer.w1, r.ends)
    dw2 = dg.gemm_tn_grouped(dy, h, r.ends)
    dw1, db1 = dg.gemm_tn_grouped(dz, xs, r.ends, colsum=True)
    for e, lo, hi in _layer.spans(r.ends.tolist()):
        if lo < hi:
            _layer.check_forward(h[lo:hi], z[lo:hi], xs[lo:hi], layer.w1[e], "nt", layer.b1[e], "silu", None, "first")
            _layer.check_dact(dz[lo:hi], dy[lo:hi], layer.w2[e], "nn", z[lo:hi], "silu", "dz")
            _layer.check_tn(dw2[e], None, dy[lo:hi], h[lo:hi], "dw2")
            _layer.check_tn(dw1[e], db1[e], dz[lo:hi], xs[lo:hi], "dw1")
    # the gathered rows' gradient: each token's choices added up, and the skip's
    dx = dg.combine_rows(dxs, r.places, residual=dout)
    _experts.check_combine(dx, dxs, r.places, None, dout, "dx")
    score, renorm = layer.routing.get("score", "softmax"), layer.routing.get("renorm", True)
    dl = dg.route_grad(l, r.experts, dw, score=score, renorm=renorm)
    _experts.check_route_grad(dl, l, r.experts, dw, score, renorm, 1.0, "dlogits")
    dx2 = dg.gemm_nn_fused(dl, layer.router, residual=dx)
    _layer.check_forward(dx2, None, dl, layer.router, "nn", None, "none", dx, "dx")


def test_a_training_step_in_a_graph():
    E, N, F, dtype, kw = CONFIGS[0]
    layer = Layer(E, N, F, dtype, **kw)
    x, dout = tokens(200, N, dtype), tokens(200, N, dtype, seed=9)
    dh = torch.zeros((200 * layer.k, N), dtype=dtype, device="cuda")

    def step():
        l = layer.logits(x)
        r = dg.route(l, layer.k, **layer.routing)
        xs = x.index_select(0, r.tokens)
        z = torch.zeros((200 * layer.k, F), dtype=dtype, device="cuda")
        h = dg.gemm_nt_grouped(xs, layer.w1, r.ends, bias=layer.b1, act="silu", preact=z)
        y = dg.gemm_nt_grouped(h, layer.w2, r.ends)
        out = dg.combine_rows(y, r.places, r.weights, residual=x)
        dy, dw = dg.combine_rows_grad(dout, y, r.places, r.weights, dh=dh)
        dl = dg.route_grad(l, r.experts, dw)
        dxs = dg.gemm_nn_grouped(dg.gemm_nn_grouped_dact(dy, layer.w2, r.ends, z, "silu"), layer.w1, r.ends)
        return out, dw, dl, dg.combine_rows(dxs, r.places, residual=dout), dg.gemm_tn_grouped(dy, h, r.ends)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(4):
        x.copy_(tokens(200, N, dtype, seed=20 + rep))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
