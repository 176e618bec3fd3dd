"""The operators of an expert layer around its products, and of its products
in 8-bit integers, as measured cases.

* ``route``         router logits to the experts of every token: scores, a
                    balance bias, groups, top-k, weights; and the dispatch:
                    the experts' ends, the token of each sorted row and the
                    sorted row of each choice;
* ``route_grad``    the gradient of the logits from that of the weights;
* ``quantize``      rows to int8 with a scale each, gathered by token where
                    they are dispatched to experts;
* ``i8``            D = act((A.B^T) sa sb + bias) + residual with A, B in
                    int8, a scale per row of A and per row of B;
* ``i8_grouped``    the same for rows sorted by expert;
* ``combine``       the experts' rows back to their tokens: weighted sums,
                    with the skip connection;
* ``combine_grad``  its gradients: the experts' rows and the weights.

Rows sorted by expert are described by ``ends``, the running sum of the
experts' row counts; rows at or past the last end belong to nobody.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a decoding batch: a few tokens over 64 experts, two each; the call
        # whose latency counts
        dict(name="route_tokens", op="route", dtype="bf16", T=16, E=64, k=2, score="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.0),
        # a training step's tokens over many experts in groups, with a bias
        # that balances their loads
        dict(name="route_train", op="route", dtype="f32", T=16384, E=256, k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # the gradient through an odd number of experts and tokens, weights
        # that are not renormalised: dense rows
        dict(name="route_grad_odd", op="route_grad", dtype="bf16", T=20011, E=48, k=6,
             score="softmax", renorm=False, scale=1.0),
        # one token's activations, before a projection in int8
        dict(name="quantize_token", op="quantize", dtype="bf16", T=1, K=4096, k=0, pad=0),
        # a batch's tokens sent to two experts each, quantised on the way; the
        # batch is padded
        dict(name="quantize_dispatch", op="quantize", dtype="bf16", T=8192, K=4096, k=2, pad=300),
        # one token of a decoder through a gate or up projection
        dict(name="i8_token", op="i8", dtype="bf16", M=1, N=4096, K=4096, bias=True, act="silu",
             residual=False, preact=False),
        # sizes that divide no tile, the pre-activation kept
        dict(name="i8_ragged", op="i8", dtype="f16", M=3000, N=5000, K=4000, bias=True, act="gelu",
             residual=False, preact=True),
        # a prefill's down projection with the skip connection: the largest
        dict(name="i8_large", op="i8", dtype="bf16", M=8192, N=5120, K=17408, bias=False,
             act="none", residual=True, preact=False),
        # a decoding batch of a few sequences, two experts for each token: one
        # pass over the weights of the experts that were chosen
        dict(name="i8_experts_tokens", op="i8_grouped", dtype="bf16", G=64, rows=32, active=24,
             skew=0.5, pad=0, N=2048, K=2048, bias=False, act="silu", residual=False, preact=False),
        # a prefill's tokens over sixteen experts, unevenly loaded
        dict(name="i8_experts_prefill", op="i8_grouped", dtype="bf16", G=16, rows=16384, active=16,
             skew=0.5, pad=120, N=4096, K=4096, bias=True, act="gelu_tanh", residual=False,
             preact=False),
        # the experts' rows of an odd batch back to its tokens
        dict(name="combine_ragged", op="combine", dtype="f16", T=777, N=1001, k=3, weights=True,
             residual=True, missing=0.05),
        # its gradients in a training step
        dict(name="combine_grad_train", op="combine_grad", dtype="bf16", T=8192, N=4096, k=2,
             weights=True, missing=0.0),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 64 or of 8,
    or any number."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    step = rng.choice((64, 8, 1))
    return int(min(hi, max(lo, round(x / step) * step)))


def draw(rng):
    most = [work(c) for c in listed()]
    flops, moved = max(w["flops"] for w in most), max(w["bytes"] for w in most)
    while True:
        op = rng.choice(("route", "route", "route_grad", "quantize", "i8", "i8", "i8_grouped",
                         "i8_grouped", "combine", "combine_grad"))
        case = dict(op=op, dtype=rng.choice(("f16", "bf16")))
        if op.startswith("route"):
            case["dtype"] = rng.choice(("f32", "f16", "bf16"))
            groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
            E = groups * _size(rng, 4, 512 // groups)
            case.update(T=_size(rng, 1, 32768), E=E, score=rng.choice(("softmax", "sigmoid")),
                        renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)))
            kept = E
            if op == "route":
                top = rng.randint(1, groups)
                kept = E // groups * top
                case.update(bias=rng.random() < 0.5, groups=groups, top_groups=top,
                            group_top=rng.choice((1, 2)), masked=rng.choice((0.0, 0.0, 0.1)))
            case["k"] = rng.randint(1, min(10, kept))
        elif op == "quantize":
            k = rng.choice((0, 0, 1, 2, 6))
            case.update(T=_size(rng, 1, 16384), K=_size(rng, 16, 17408), k=k,
                        pad=rng.randint(0, 300) if k else 0)
        elif op.startswith("i8"):
            if op == "i8":
                case.update(M=_size(rng, 1, 16384), N=_size(rng, 16, 18000), K=_size(rng, 16, 18000))
            else:
                G = _size(rng, 2, 128)
                active = rng.randint(max(1, G // 3), G)
                case.update(G=G, rows=_size(rng, active, 16384), active=active,
                            skew=rng.choice((0.5, 1.0)), pad=rng.choice((0, 0, rng.randint(1, 300))),
                            N=_size(rng, 32, 5000), K=_size(rng, 32, 5000))
            case.update(bias=rng.random() < 0.6, act=rng.choice(_ACTS),
                        residual=rng.random() < 0.4, preact=rng.random() < 0.3)
            if case.get("G", 1) * case["N"] * case["K"] > 3 << 29:
                continue
        else:
            case.update(T=_size(rng, 1, 16384), N=_size(rng, 16, 8192), k=rng.randint(1, 8),
                        weights=op == "combine_grad" or rng.random() < 0.8,
                        missing=rng.choice((0.0, 0.0, 0.1)))
            if op == "combine":
                case["residual"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] <= flops and w["bytes"] <= moved:
            return case


# ----------------------------------------------------------------- inputs --

def _group_sizes(case, seed):
    """Row counts of the G experts: `active` of them, picked at random, share
    the rows in uneven parts of at least one row each."""
    rng = np.random.default_rng([seed, 78])
    sizes = np.zeros(case["G"], dtype=np.int64)
    who = rng.permutation(case["G"])[:case["active"]]
    share = rng.exponential(size=case["active"]) ** case["skew"] + 1e-3
    sizes[who] = 1 + rng.multinomial(case["rows"] - case["active"], share / share.sum())
    return [int(s) for s in sizes]


def prepare(case, seed):
    dt = _DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    op = case["op"]
    st = dict(case=case)

    def normal(shape, sigma, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def codes(*shape):
        # int8 values as quantised activations and weights have them, drawn in
        # pieces: a stack of weights in 32 bits would not be small
        out = torch.empty(shape, dtype=torch.int8, device="cuda")
        flat = out.view(-1)
        for lo in range(0, flat.numel(), 1 << 28):
            part = flat[lo:lo + (1 << 28)]
            part.copy_((torch.randn(part.numel(), generator=gen, device="cuda") * 32)
                       .round_().clamp_(-127, 127))
        return out

    def scales(*shape):
        return torch.exp(torch.randn(shape, generator=gen, device="cuda") * 0.2) / 32

    if op == "route":
        T, E = case["T"], case["E"]
        st["logits"] = normal((T, E), 1.5)
        if case["masked"]:
            # experts that are switched off, and tokens that are padding
            st["logits"][:, uniform(E) < case["masked"]] = -math.inf
            st["logits"][uniform(T) < case["masked"]] = -math.inf
        st["bias"] = normal((E,), 0.1, torch.float32) if case["bias"] else None
    elif op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = normal((T, E), 1.5)
        st["experts"] = torch.sort(st["logits"].float(), dim=1, descending=True,
                                   stable=True).indices[:, :k].to(torch.int32).contiguous()
        st["dweights"] = normal((T, k), 1.0, torch.float32)
    elif op == "quantize":
        T, k = case["T"], case["k"]
        # activations: a normal bulk, and rows of different sizes
        st["x"] = (torch.randn((T, case["K"]), generator=gen, device="cuda") *
                   torch.exp(torch.randn((T, 1), generator=gen, device="cuda"))).to(dt)
        st["rows"] = None
        if k:
            # the tokens of the sorted rows: each k times, in the experts' order;
            # the rows behind the last expert's have none
            order = torch.randperm(T * k, generator=gen, device="cuda") // k
            st["rows"] = torch.cat([order, torch.full((case["pad"],), -1, device="cuda")]).to(torch.int32)
    elif op.startswith("i8"):
        G, M = (), case.get("M")
        if op == "i8_grouped":
            sizes = _group_sizes(case, seed)
            ends = np.cumsum(sizes)
            G, M = (case["G"],), case["rows"] + case["pad"]
            st["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            st["sizes"] = sizes
        N, K = case["N"], case["K"]
        st["A"], st["SA"] = codes(M, K), scales(M)
        st["B"], st["SB"] = codes(*G, N, K), scales(*G, N) * K ** -0.5
        st["bias"] = normal(G + (N,), 0.5) if case["bias"] else None
        st["residual"] = normal((M, N), 1.0) if case["residual"] else None
        st["Z"] = torch.zeros((M, N), dtype=dt, device="cuda") if case["preact"] else None
        st["D"] = torch.zeros((M, N), dtype=dt, device="cuda")
    else:
        T, N, k = case["T"], case["N"], case["k"]
        st["h"] = normal((T * k, N), 1.0)
        places = torch.randperm(T * k, generator=gen, device="cuda").to(torch.int32).view(T, k)
        # choices that a token did not have
        st["places"] = torch.where(uniform(T, k) < case["missing"], torch.full_like(places, -1), places)
        w = uniform(T, k) + 0.05
        st["w"] = w / w.sum(1, keepdim=True) if case["weights"] else None
        if op == "combine":
            st["residual"] = normal((T, N), 1.0) if case["residual"] else None
        else:
            st["dy"] = normal((T, N), 1.0)
            st["dh"] = torch.zeros((T * k, N), dtype=dt, device="cuda")
    return st


# ----------------------------------------------- the operators, plainly ----

def _plain_route(st, case):
    # (in 64 bits: two scores may lie closer to each other than 32 bits tell)
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = st["logits"].double()
    broken = ~(l < math.inf).all(1, keepdim=True)
    if case["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        s = torch.exp(l - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    # (without a bias the scores rank as the logits do)
    c = s if st["bias"] is None else s + st["bias"].double()
    c = torch.where((l > -math.inf) & (c > -math.inf), c, torch.full_like(c, -math.inf))
    rank = c if st["bias"] is not None else l
    if case["top_groups"] < G:
        m = case["group_top"]
        of = (rank if m == 1 else c).view(T, G, E // G)
        best = torch.sort(of, dim=2, descending=True).values[:, :, :m]
        some = best[:, :, 0] > -math.inf
        value = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        value = torch.where(some, value, torch.full_like(value, -math.inf))
        first = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        stays = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, first, True)
        rank = torch.where(stays[:, :, None].expand(T, G, E // G).reshape(T, E), rank,
                           torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    e = order.indices[:, :k]
    there = (order.values[:, :k] > -math.inf) & ~broken
    w = torch.where(there, s.gather(1, e), torch.zeros((), dtype=s.dtype, device=s.device))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    w = torch.where(broken, torch.full_like(w, math.nan), w * case["scale"]).float()
    e = torch.where(there, e, torch.full_like(e, -1))
    # the dispatch: choices sorted by expert, in the tokens' order for each
    flat = torch.where(there, e, torch.full_like(e, E)).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    ends = torch.cumsum(torch.bincount(flat, minlength=E + 1)[:E], 0)
    n = torch.arange(T * k, device=l.device)
    inside = n < ends[-1]
    tokens = torch.where(inside, order // k, torch.full_like(order, -1))
    places = torch.empty_like(order)
    places[order] = torch.where(inside, n, torch.full_like(n, -1))
    i32 = torch.int32
    return (w, e.to(i32), places.view(T, k).to(i32), ends.to(i32), tokens.to(i32))


def _plain_route_grad(st, case):
    l, e, dw = st["logits"].float(), st["experts"].long(), st["dweights"]
    if case["score"] == "softmax":
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    ds = torch.zeros_like(l)
    chosen = s.gather(1, e)
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        v = chosen / total
        d = (dw - (v * dw).sum(1, keepdim=True)) / total
    else:
        d = dw
    ds.scatter_(1, e, d * case["scale"])
    if case["score"] == "softmax":
        dl = s * (ds - (s * ds).sum(1, keepdim=True))
    else:
        dl = ds * s * (1.0 - s)
    return (dl.to(st["logits"].dtype),)


def _plain_quantize(st, case):
    # (in 64 bits: a value half-way between two whole numbers has to stay there)
    x = st["x"] if st["rows"] is None else st["x"][st["rows"].long().clamp(min=0)]
    if st["rows"] is not None:
        x = torch.where((st["rows"] >= 0)[:, None], x, torch.zeros_like(x))
    x = x.double()
    most = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127.0 / torch.where(most > 0, most, torch.ones_like(most)))
    return (q.to(torch.int8), (most[:, 0] / 127.0).float())


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_i8(st, case):
    dt = st["D"].dtype

    def finish(P, rows, sb, bias):
        z = P * st["SA"][rows, None] * sb
        if bias is not None:
            z = z + bias.float()
        if st["Z"] is not None:
            st["Z"][rows] = z.to(dt)
        d = _act(z, case["act"])
        if st["residual"] is not None:
            d = d + st["residual"][rows].float()
        st["D"][rows] = d.to(dt)

    A, B, bias = st["A"], st["B"], st["bias"]
    if case["op"] == "i8":
        finish(A.float() @ B.float().t(), slice(0, case["M"]), st["SB"], bias)
    elif case["rows"] <= 16 * case["G"]:
        # few rows: each expert's padded to those of the fullest, one batched
        # product over the experts that have rows (one by one they take twice
        # as long)
        R = case["rows"]
        sizes = torch.tensor(st["sizes"], device="cuda")
        g = torch.repeat_interleave(torch.arange(case["G"], device="cuda"), sizes)
        at = torch.arange(R, device="cuda") - (st["ends"].long() - sizes)[g]
        used = torch.nonzero(sizes)[:, 0]
        slot = torch.zeros_like(sizes)
        slot[used] = torch.arange(used.numel(), device="cuda")
        a = torch.zeros((used.numel(), max(st["sizes"]), case["K"]), device="cuda")
        a[slot[g], at] = A[:R].float()
        P = torch.bmm(a, B[used].float().transpose(1, 2).contiguous())[slot[g], at]
        finish(P, slice(0, R), st["SB"][g], None if bias is None else bias[g])
    else:
        # many: expert by expert (padded to one batched product, uneven
        # experts take twice as long)
        lo = 0
        for g, n in enumerate(st["sizes"]):
            if n:
                finish(A[lo:lo + n].float() @ B[g].float().t(), slice(lo, lo + n), st["SB"][g],
                       None if bias is None else bias[g])
            lo += n
    return (st["D"],) if st["Z"] is None else (st["D"], st["Z"])


def _rows_of(h, places):
    """h's rows at the places (T x k x N, in 32 bits), zeros where there is none."""
    r = h[places.long().clamp(min=0)].float()
    return torch.where((places >= 0)[:, :, None], r, torch.zeros_like(r))


def _plain_combine(st, case):
    r = _rows_of(st["h"], st["places"])
    y = (r if st["w"] is None else r * st["w"][:, :, None]).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return (y.to(st["h"].dtype),)


def _plain_combine_grad(st, case):
    dy = st["dy"].float()
    dw = (_rows_of(st["h"], st["places"]) * dy[:, None, :]).sum(2)
    there = st["places"] >= 0
    st["dh"][st["places"][there].long()] = (st["w"][:, :, None] * dy[:, None, :])[there].to(st["dh"].dtype)
    return (st["dh"], dw)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(st, case)
    if op == "route_grad":
        return _plain_route_grad(st, case)
    if op == "quantize":
        return _plain_quantize(st, case)
    if op.startswith("i8"):
        return _plain_i8(st, case)
    return _plain_combine(st, case) if op == "combine" else _plain_combine_grad(st, case)


# --------------------------------------- the operators, by the library -----

def _own(st):
    import dense_gemm_08_amd as dg
    case = st["case"]
    op = case["op"]
    if op == "route":
        r = dg.route(st["logits"], case["k"], score=case["score"], bias=st["bias"],
                     groups=case["groups"], top_groups=case["top_groups"],
                     group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
        return (r.weights, r.experts, r.places, r.ends, r.tokens)
    if op == "route_grad":
        return (dg.route_grad(st["logits"], st["experts"], st["dweights"], score=case["score"],
                              renorm=case["renorm"], scale=case["scale"]),)
    if op == "quantize":
        return dg.quantize_rows(st["x"], rows=st["rows"])
    if op == "combine":
        return (dg.combine_rows(st["h"], st["places"], st["w"], residual=st["residual"]),)
    if op == "combine_grad":
        return dg.combine_rows_grad(st["dy"], st["h"], st["places"], st["w"], dh=st["dh"])
    kw = dict(bias=st["bias"], act=case["act"], residual=st["residual"], preact=st["Z"], D=st["D"])
    if op == "i8":
        d = dg.gemm_nt_i8(st["A"], st["SA"], st["B"], st["SB"], **kw)
    else:
        d = dg.gemm_nt_i8_grouped(st["A"], st["SA"], st["B"], st["SB"], st["ends"], **kw)
    return (d,) if st["Z"] is None else (d, st["Z"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    """Each input read once, each output written once (of the experts' weights,
    those that have rows); two operations for each multiplication and addition
    of a product, a few for each logit, element and choice elsewhere."""
    op = case["op"]
    wide = 4 if case["dtype"] == "f32" else 2
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": wide * T * E + 4 * E * (1 + case["bias"]) + 16 * T * k, "flops": 4 * T * E}
    if op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 2 * wide * T * E + 8 * T * k, "flops": 6 * T * E}
    if op == "quantize":
        T, K, R = case["T"], case["K"], case["T"] * max(case["k"], 1) + case["pad"]
        return {"bytes": 2 * T * K + R * (K + 4) + (4 * R if case["k"] else 0), "flops": 4 * R * K}
    if op.startswith("combine"):
        T, N, k = case["T"], case["N"], case["k"]
        if op == "combine":
            rows = T * k + T + (T if case["residual"] else 0)
            return {"bytes": 2 * rows * N + T * k * (4 + 4 * case["weights"]), "flops": 2 * T * k * N}
        return {"bytes": 2 * (2 * T * k + T) * N + 12 * T * k, "flops": 3 * T * k * N}
    R = case["rows"] if op == "i8_grouped" else case["M"]
    G = case["active"] if op == "i8_grouped" else 1
    N, K = case["N"], case["K"]
    moved = R * (K + 4) + G * N * (K + 4) + 2 * R * N * (1 + case["residual"] + case["preact"])
    moved += 2 * G * N if case["bias"] else 0
    return {"bytes": moved + 4 * case.get("G", 0), "flops": 2 * R * N * K}


# ------------------------------------------------------ the exact results --

def _exact_route(st, case):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = st["logits"].double().cpu().numpy()
    b = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    with np.errstate(all="ignore"):
        on = l > -np.inf
        if case["score"] == "softmax":
            top = np.max(l, axis=1, keepdims=True)
            p = np.where(on, np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
            s = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        else:
            s = np.where(on, np.exp(-np.logaddexp(0.0, -l)), 0.0)
        c = s + (0.0 if b is None else b)
        key = np.where(on, l if b is None else c, -np.inf)
        if case["top_groups"] < G:
            use = key if case["group_top"] == 1 else np.where(on, c, -np.inf)
            of = -np.sort(-use.reshape(T, G, E // G), axis=2)[:, :, :case["group_top"]]
            value = np.where(np.isfinite(of[:, :, 0]), np.where(np.isfinite(of), of, 0.0).sum(axis=2), -np.inf)
            rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
            key = np.where(np.repeat(rank < case["top_groups"], E // G, axis=1), key, -np.inf)
        e = np.argsort(-key, axis=1, kind="stable")[:, :k]
        there = np.isfinite(np.take_along_axis(key, e, axis=1))
        w = np.where(there, np.take_along_axis(s, e, axis=1), 0.0)
        if case["renorm"]:
            w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return (torch.from_numpy(w * case["scale"]), None, None, None, None)


def _exact_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        # 0.5 (1 + tanh u) is the logistic function of 2 u
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z * z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st, case)
    if op == "route_grad":
        l, e, dw = st["logits"].double(), st["experts"].long(), st["dweights"].double()
        scale = case["scale"]
        picked = l.gather(1, e)
        if case["renorm"]:
            # the weights' own gradient, at the chosen logits alone
            lw = picked if case["score"] == "softmax" else torch.nn.functional.logsigmoid(picked)
            v = torch.softmax(lw, dim=1)
            d = scale * v * (dw - (v * dw).sum(dim=1, keepdim=True))
            if case["score"] == "sigmoid":
                d = d * torch.sigmoid(-picked)
            return (torch.zeros_like(l).scatter_add_(1, e, d),)
        if case["score"] == "sigmoid":
            return (torch.zeros_like(l).scatter_add_(1, e, scale * dw * torch.sigmoid(picked) *
                                                     torch.sigmoid(-picked)),)
        p = torch.softmax(l, dim=1)
        mean = (p.gather(1, e) * dw).sum(dim=1, keepdim=True)
        return (scale * (torch.zeros_like(l).scatter_add_(1, e, p.gather(1, e) * dw) - p * mean),)
    if op == "quantize":
        x = st["x"].double()
        most = x.abs().max(dim=1).values / 127.0
        if st["rows"] is None:
            return (None, most)
        at = st["rows"].long()
        return (None, torch.where(at < 0, torch.zeros((), dtype=torch.float64, device="cuda"), most[at]))
    if op == "combine":
        y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        if st["residual"] is not None:
            y += st["residual"].double()
        for j in range(case["k"]):
            at = st["places"][:, j].long()
            f = (at >= 0).double() if st["w"] is None else st["w"][:, j].double() * (at >= 0)
            y += f[:, None] * st["h"][at.clamp(min=0)].double()
        return (y,)
    if op == "combine_grad":
        dy = st["dy"].double()
        dh = torch.zeros(st["h"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(st["places"].shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = torch.nonzero(st["places"][:, j] >= 0)[:, 0]
            at = st["places"][t, j].long()
            dh[at] = st["w"][t, j].double()[:, None] * dy[t]
            dw[t, j] = torch.linalg.vecdot(dy[t], st["h"][at].double())
        return (dh, dw)
    bounds = [(None, 0, case["M"])] if op == "i8" else [
        (g, int(e) - n, int(e)) for g, (e, n) in enumerate(zip(np.cumsum(st["sizes"]), st["sizes"]))]
    D = torch.zeros(st["D"].shape, dtype=torch.float64, device="cuda")
    Z = torch.zeros_like(D)
    for g, lo, hi in bounds:
        if lo == hi:
            continue
        B, sb, bias = [None if x is None else x if g is None else x[g]
                       for x in (st["B"], st["SB"], st["bias"])]
        z = torch.mm(st["A"][lo:hi].double() * st["SA"][lo:hi].double()[:, None],
                     (B.double() * sb.double()[:, None]).t())
        if bias is not None:
            z = z + bias.double()
        Z[lo:hi] = z
        D[lo:hi] = _exact_act(z, case["act"])
        if st["residual"] is not None:
            D[lo:hi] += st["residual"][lo:hi].double()
    return (D,) if st["Z"] is None else (D, Z)
