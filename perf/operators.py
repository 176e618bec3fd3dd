"""The operators of a transformer's dense and expert layers, as measured cases.

Three products and their gradients, next to the library's plain ones:

* ``fused``         D = act(A.B + bias) + residual, Z = A.B + bias kept where
                    a backward pass will need it (one layer, forward);
* ``dact``          D = (A.B) * act'(Z): the gradient that a layer hands back
                    through the activation below it;
* ``tn``            D = A^T.B with the column sums of A: a layer's weight and
                    bias gradients, the sum running over the tokens;
* ``grouped``       the first product for rows sorted by expert, each expert
                    with a weight matrix and a bias of its own;
* ``grouped_dact``  the second for rows sorted by expert;
* ``grouped_tn``    the third per expert: the sum runs over the expert's rows.

B is N x K for the layout "nt" and K x N for "nn" (a stack of such matrices
for the grouped products).  Rows sorted by expert are described by ``ends``,
the running sum of the experts' row counts; rows at or past the last end
belong to nobody and keep what they held.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_GRAD_ACTS = ("relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decoder through a gate or up projection: the call
        # whose latency counts, bounded by one pass over the weights
        dict(name="fused_token", op="fused", dtype="bf16", layout="nt", M=1, N=4096, K=4096,
             bias=True, act="silu", residual=False, preact=False),
        # a training step's first projection on sizes that divide no tile,
        # the pre-activation kept for the backward pass
        dict(name="fused_ragged", op="fused", dtype="f16", layout="nt", M=3000, N=5000, K=4000,
             bias=True, act="gelu", residual=False, preact=True),
        # a prefill's down projection with the skip connection added: the
        # largest product
        dict(name="fused_large", op="fused", dtype="bf16", layout="nn", M=8192, N=5120, K=17408,
             bias=True, act="none", residual=True, preact=False),
        # the gradient through a down projection and the activation below it
        dict(name="dact_square", op="dact", dtype="bf16", layout="nn", M=4096, N=4096, K=4096,
             act="gelu_tanh"),
        # the same on odd sizes, whose rows are not 16-byte aligned
        dict(name="dact_odd", op="dact", dtype="f16", layout="nt", M=777, N=1001, K=2051,
             act="silu"),
        # the weight and bias gradient of a wide projection over a batch's tokens
        dict(name="tn_large", op="tn", dtype="bf16", M=5120, N=8192, K=8192, colsum=True),
        # the same for a narrow projection over a long, odd number of tokens:
        # few output tiles, a long sum
        dict(name="tn_narrow", op="tn", dtype="f16", M=512, N=640, K=20011, colsum=True),
        # a decoding batch of a few sequences, two experts for each token:
        # one pass over the weights of the experts that were chosen
        dict(name="grouped_tokens", op="grouped", dtype="bf16", layout="nt", G=64, rows=32,
             active=24, skew=1.0, pad=0, N=2048, K=2048, bias=True, act="silu", residual=False,
             preact=False),
        # a training step's tokens over sixteen experts, unevenly loaded, the
        # pre-activation kept
        dict(name="grouped_train", op="grouped", dtype="bf16", layout="nt", G=16, rows=16384,
             active=16, skew=2.0, pad=0, N=4096, K=4096, bias=True, act="gelu_tanh",
             residual=False, preact=True),
        # the gradient to the experts' inputs: many experts, some of them
        # idle, and a batch padded past its last token
        dict(name="grouped_dact_ragged", op="grouped_dact", dtype="f16", layout="nn", G=48,
             rows=5003, active=41, skew=1.0, pad=117, N=1400, K=1000, act="silu"),
        # the experts' weight and bias gradients of that training step
        dict(name="grouped_tn_train", op="grouped_tn", dtype="bf16", G=16, rows=16384, active=16,
             skew=2.0, pad=0, M=4096, N=4096, colsum=True),
        # many small experts, some idle, on odd sizes
        dict(name="grouped_tn_odd", op="grouped_tn", dtype="f16", G=40, rows=3001, active=33,
             skew=1.0, pad=64, M=520, N=1001, colsum=False),
    ]


def _cost(case):
    return work(case)["flops"]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: a multiple of 64 or of 8,
    or any number."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    step = rng.choice((64, 8, 1))
    return int(min(hi, max(lo, round(x / step) * step)))


def draw(rng):
    cap = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("fused", "dact", "tn", "grouped", "grouped_dact", "grouped_tn"))
        case = dict(op=op, dtype=rng.choice(("f16", "bf16")))
        if not op.endswith("tn"):
            case["layout"] = rng.choice(("nt", "nn"))
        if op.startswith("grouped"):
            G = _size(rng, 2, 160)
            active = rng.randint(max(1, G // 3), G)
            rows = _size(rng, active, 24000)
            case.update(G=G, rows=rows, active=active, skew=rng.choice((0.5, 1.0, 2.0)),
                        pad=rng.choice((0, 0, rng.randint(1, 300))))
            sizes = (_size(rng, 32, 6000), _size(rng, 32, 6000))
        elif op == "tn":
            case["K"] = _size(rng, 1, 32000)
            sizes = (_size(rng, 16, 18000), _size(rng, 16, 18000))
        else:
            case["M"] = _size(rng, 1, 16384)
            sizes = (_size(rng, 16, 18000), _size(rng, 16, 18000))
        if op.endswith("tn"):
            case.update(M=sizes[0], N=sizes[1], colsum=rng.random() < 0.6)
        else:
            case.update(N=sizes[0], K=sizes[1])
            if op.endswith("dact"):
                case["act"] = rng.choice(_GRAD_ACTS)
            else:
                case.update(bias=rng.random() < 0.7, act=rng.choice(_ACTS),
                            residual=rng.random() < 0.5, preact=rng.random() < 0.4)
        grouped_bytes = 2 * case.get("G", 1) * sizes[0] * sizes[1]
        if _cost(case) <= cap and grouped_bytes <= 3 << 30:
            return case


# ----------------------------------------------------------------- inputs --

def _group_sizes(case, seed):
    """Row counts of the G experts: `active` of them, picked at random, share
    the rows in uneven parts of at least one row each."""
    rng = np.random.default_rng([seed, 77])
    sizes = np.zeros(case["G"], dtype=np.int64)
    who = rng.permutation(case["G"])[:case["active"]]
    share = rng.exponential(size=case["active"]) ** case["skew"] + 1e-3
    spare = case["rows"] - case["active"]
    sizes[who] = 1 + rng.multinomial(spare, share / share.sum())
    return [int(s) for s in sizes]


def prepare(case, seed):
    dt = _DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)

    def normal(shape, sigma):
        # (drawn in pieces: a stack of weights in 32 bits would not be small)
        out = torch.empty(shape, dtype=dt, device="cuda")
        flat = out.view(-1)
        for lo in range(0, flat.numel(), 1 << 28):
            part = flat[lo:lo + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=gen, device="cuda") * sigma)
        return out

    op = case["op"]
    st = dict(case=case)
    if op.startswith("grouped"):
        sizes = _group_sizes(case, seed)
        st["sizes"] = sizes
        st["ends"] = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
        G, R = (case["G"],), case["rows"] + case["pad"]
    else:
        G, R = (), case.get("M")
    if op.endswith("tn"):
        # the gradient of a layer's output and the layer's input, one row a token
        T = R if op == "grouped_tn" else case["K"]
        st["A"] = normal((T, case["M"]), 1.0)
        st["B"] = normal((T, case["N"]), 1.0)
        return st
    N, K = case["N"], case["K"]
    st["A"] = normal((R, K), 1.0)
    st["B"] = normal(G + ((N, K) if case["layout"] == "nt" else (K, N)), K ** -0.5)
    if op.endswith("dact"):
        st["Z"] = normal((R, N), 1.0)
    else:
        st["bias"] = normal(G + (N,), 0.5) if case["bias"] else None
        st["residual"] = normal((R, N), 1.0) if case["residual"] else None
        st["Z"] = torch.zeros((R, N), dtype=dt, device="cuda") if case["preact"] else None
    st["D"] = torch.zeros((R, N), dtype=dt, device="cuda")
    return st


# ----------------------------------------------- the operators, plainly ----

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


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        pdf = torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * pdf
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _product(a, b, layout):
    return a.float() @ (b.float().t() if layout == "nt" else b.float())


def _plain_rows(st, case, rows, g):
    """The rows `rows` (a slice) of a fused or dact product, with expert g's
    matrix and bias (g None: the one there is)."""
    b = st["B"] if g is None else st["B"][g]
    z = _product(st["A"][rows], b, case["layout"])
    if case["op"].endswith("dact"):
        st["D"][rows] = (z * _act_grad(st["Z"][rows].float(), case["act"])).to(st["D"].dtype)
        return
    if st["bias"] is not None:
        z = z + (st["bias"] if g is None else st["bias"][g]).float()
    if st["Z"] is not None:
        st["Z"][rows] = z.to(st["Z"].dtype)
    d = _act(z, case["act"])
    if st["residual"] is not None:
        d = d + st["residual"][rows].float()
    st["D"][rows] = d.to(st["D"].dtype)


def _plain(st):
    case = st["case"]
    op = case["op"]
    dt = st["A"].dtype
    if op == "tn":
        a = st["A"].float()
        d = (a.t() @ st["B"].float()).to(dt)
        return (d, a.sum(0).to(dt)) if case["colsum"] else (d,)
    if op == "grouped_tn":
        G, M, N = case["G"], case["M"], case["N"]
        d = torch.zeros((G, M, N), dtype=dt, device="cuda")
        c = torch.zeros((G, M), dtype=dt, device="cuda") if case["colsum"] else None
        lo = 0
        for g, n in enumerate(st["sizes"]):
            if n:
                a = st["A"][lo:lo + n].float()
                d[g] = (a.t() @ st["B"][lo:lo + n].float()).to(dt)
                if c is not None:
                    c[g] = a.sum(0).to(dt)
            lo += n
        return (d,) if c is None else (d, c)
    if op.startswith("grouped"):
        lo = 0
        for g, n in enumerate(st["sizes"]):
            if n:
                _plain_rows(st, case, slice(lo, lo + n), g)
            lo += n
    else:
        _plain_rows(st, case, slice(0, case["M"]), None)
    if op.endswith("dact") or st["Z"] is None:
        return (st["D"],)
    return (st["D"], st["Z"])


# --------------------------------------- the operators, by the library -----

def _own(st):
    import dense_gemm_08_amd as dg
    case = st["case"]
    op = case["op"]
    if op == "tn":
        if case["colsum"]:
            return dg.gemm_tn(st["A"], st["B"], colsum=True)
        return (dg.gemm_tn(st["A"], st["B"]),)
    if op == "grouped_tn":
        if case["colsum"]:
            return dg.gemm_tn_grouped(st["A"], st["B"], st["ends"], colsum=True)
        return (dg.gemm_tn_grouped(st["A"], st["B"], st["ends"]),)
    nt = case["layout"] == "nt"
    if op == "dact":
        f = dg.gemm_nt_dact if nt else dg.gemm_nn_dact
        return (f(st["A"], st["B"], st["Z"], case["act"], D=st["D"]),)
    if op == "grouped_dact":
        f = dg.gemm_nt_grouped_dact if nt else dg.gemm_nn_grouped_dact
        return (f(st["A"], st["B"], st["ends"], st["Z"], case["act"], D=st["D"]),)
    if op == "fused":
        f = dg.gemm_nt_fused if nt else dg.gemm_nn_fused
        d = f(st["A"], st["B"], bias=st["bias"], act=case["act"], residual=st["residual"],
              preact=st["Z"], D=st["D"])
    else:
        f = dg.gemm_nt_grouped if nt else dg.gemm_nn_grouped
        d = f(st["A"], st["B"], st["ends"], bias=st["bias"], act=case["act"],
              residual=st["residual"], preact=st["Z"], D=st["D"])
    return (d,) if st["Z"] is None else (d, st["Z"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --

def work(case):
    """Each input read once, each output written once (of the experts, those
    that have rows; a gradient is written for every expert); two operations
    for each multiplication and addition of the products."""
    op = case["op"]
    grouped = op.startswith("grouped")
    if op.endswith("tn"):
        T = case["rows"] if grouped else case["K"]
        G = case["G"] if grouped else 1
        M, N = case["M"], case["N"]
        elems = T * (M + N) + G * M * N + (G * M if case["colsum"] else 0)
        return {"bytes": 2 * elems + (4 * G if grouped else 0), "flops": 2 * T * M * N}
    R = case["rows"] if grouped else case["M"]
    G = case["active"] if grouped else 1
    N, K = case["N"], case["K"]
    elems = R * K + G * N * K + R * N
    if op.endswith("dact"):
        elems += R * N
    else:
        elems += (G * N if case["bias"] else 0) + R * N * (int(case["residual"]) + int(case["preact"]))
    return {"bytes": 2 * elems + (4 * case["G"] if grouped else 0), "flops": 2 * R * N * K}


# ------------------------------------------------------ the exact results --

def _phi(x):
    """The standard normal distribution function in 64 bits."""
    return torch.special.ndtr(x)


def _exact_values(z, act):
    """act(z) in 64 bits."""
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * _phi(z)
    if act == "gelu_tanh":
        # 0.5 (1 + tanh u) is the logistic function of 2 u
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z * z))
    return z * torch.sigmoid(z)


def _exact_slopes(z, act):
    """act'(z) in 64 bits."""
    if act == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act == "gelu":
        return _phi(z) + z * torch.exp(-z.square() / 2.0) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        k = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(k * z * (1.0 + 0.044715 * z * z))
        return s + z * s * (1.0 - s) * k * (1.0 + 0.134145 * z * z)
    s = torch.sigmoid(z)
    return s + z * s * (1.0 - s)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    A = st["A"].double()
    if op == "tn":
        D = torch.mm(A.t(), st["B"].double())
        return (D, A.sum(dim=0)) if case["colsum"] else (D,)
    if "sizes" in st:
        bounds = [0] + np.cumsum(st["sizes"]).tolist()
        spans = [(g, bounds[g], bounds[g + 1]) for g in range(case["G"])]
    else:
        spans = [(None, 0, case["M"])]
    if op == "grouped_tn":
        D = torch.stack([torch.mm(A[a:b].t(), st["B"][a:b].double()) if b > a else
                         torch.zeros((case["M"], case["N"]), dtype=torch.float64, device="cuda")
                         for _, a, b in spans])
        if not case["colsum"]:
            return (D,)
        return (D, torch.stack([A[a:b].sum(dim=0) for _, a, b in spans]))
    R = A.shape[0]
    D = torch.zeros((R, case["N"]), dtype=torch.float64, device="cuda")
    Z = torch.zeros_like(D)
    for g, a, b in spans:
        if a == b:
            continue
        W = (st["B"] if g is None else st["B"][g]).double()
        P = torch.mm(A[a:b], W.t() if case["layout"] == "nt" else W)
        if op.endswith("dact"):
            D[a:b] = P * _exact_slopes(st["Z"][a:b].double(), case["act"])
            continue
        if st["bias"] is not None:
            P += (st["bias"] if g is None else st["bias"][g]).double()
        Z[a:b] = P
        D[a:b] = _exact_values(P, case["act"])
        if st["residual"] is not None:
            D[a:b] += st["residual"][a:b].double()
    if op.endswith("dact") or st["Z"] is None:
        return (D,)
    return (D, Z)
