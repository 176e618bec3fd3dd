"""References and error bounds for the int8 products, routing, quantised and
combined rows: 64-bit plain forms, sharing no code with the library.

Bounds.  u = 2^-24 is half a step of FP32; a result of type t is rounded by half
a step of t (``_layer.rounding``).
* int8 products: P is exact; P sa sb is rounded three times (P to FP32, two
  products), so e = 3 u |P sa sb| (1 + 2^-20), plus u |Z| for the bias; the
  activation and the rest as for 16-bit operands (``_layer``).
* A softmax or logistic score of a chosen logit l: the difference l - m is rounded
  by u |l - m|, which moves its exponential by that relative amount; the
  exponential is within 2 u of its value, 1 + e and a division round by u each.
  So 2^-22 + u |l - m| relative.  A sum over E scores adds its additions, at most
  E / 16 + 8 in a row, and the scores' own errors, by the hardware's exponential:
  2^-22 + 1.5 u |l - m|, whose mean over the sum is below 2^-22 + 1.5 u max |l - m|.
* w_j = s_j / sum_i s_i * scale: both errors, k + 2 roundings.
"""
from __future__ import annotations

import math

import torch

from tests import _layer

U = _layer.U


# ---- int8 ------------------------------------------------------------------

def check_i8(D, Z, A, SA, B, SB, bias, act, residual, what):
    """D (and Z, unless None) against the forward epilogue of int8 A, B, whose
    product is formed exactly in 64-bit floats (below 2^53)."""
    P = A.double() @ B.double().t().contiguous()
    q = P * SA.double()[:, None] * SB.double()
    e = 3 * U * 1.000001 * q.abs()
    z = q if bias is None else q + bias.double()
    e = e + U * z.abs()
    if Z is not None:
        _layer.assert_close(Z, z, (e + _layer.rounding(z, Z.dtype)) * 1.01, what + " Z")
    d = _layer.act64(z, act)
    if act != "none":
        e = 1.13 * e + 2.0 ** -15 * d.abs() + 2.0 ** -22 * z.abs()
    if residual is not None:
        d = d + residual.double()
        e = e + U * d.abs()
    _layer.assert_close(D, d, (e + _layer.rounding(d, D.dtype)) * 1.01, what + " D")


def quantized(x):
    """(Q, S) of a matrix, by the definition: in 64 bits a half-way quotient (of
    18 by 11 bits) is itself, and all others are far from half-way."""
    x = x.double().cpu()
    m = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    bad = ~torch.isfinite(x).all(1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.bool)
    safe = torch.where((m > 0) & ~bad, m, torch.ones_like(m))
    q = torch.round(torch.where(bad[:, None], torch.zeros_like(x), x) * 127 / safe[:, None])
    s = torch.where(bad, torch.full_like(m, math.nan), m / 127).float()
    return q.to(torch.int8), s


# ---- routing ---------------------------------------------------------------

def routed(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0):
    """(weights, experts, places, ends, tokens, bound of the weights) in 64 bits,
    token by token."""
    l = logits.double().cpu()
    T, E = l.shape
    b = None if bias is None else bias.double().cpu()
    broken = ~(l < math.inf).all(1)
    lz = torch.where(broken[:, None], torch.zeros_like(l), l)
    if score == "softmax":
        top = lz.amax(1, keepdim=True)
        top = torch.where(top > -math.inf, top, torch.zeros_like(top))
        p = torch.exp(lz - top)
        s = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        far = torch.where(lz > -math.inf, top - lz, torch.zeros_like(lz))
    else:
        s = torch.sigmoid(lz)
        far = torch.zeros_like(lz)
    c = s if b is None else s + b
    on = (lz > -math.inf) & (c > -math.inf)
    key = torch.where(on, lz if b is None else c, torch.full_like(c, -math.inf))
    value = torch.where(on, c if group_top > 1 else key, torch.full_like(c, -math.inf))
    if top_groups < groups:
        size = E // groups
        best = torch.sort(value.view(T, groups, size), dim=2, descending=True).values[:, :, :group_top]
        v = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        v = torch.where(best[:, :, 0] > -math.inf, v, torch.full_like(v, -math.inf))
        order = torch.sort(v, dim=1, descending=True, stable=True).indices
        stays = torch.zeros((T, groups), dtype=torch.bool)
        stays.scatter_(1, order[:, :top_groups], True)
        key = torch.where(stays.repeat_interleave(size, dim=1), key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True)
    e = order.indices[:, :k]
    there = (order.values[:, :k] > -math.inf) & ~broken[:, None]
    lc = torch.where(there, lz.gather(1, e), torch.full((), -math.inf, dtype=torch.float64))
    if renorm:
        # with the largest chosen one's factor left out: no 0 / 0
        ls = lc if score == "softmax" else torch.nn.functional.logsigmoid(lc)
        m = ls.amax(1, keepdim=True)
        w = torch.exp(ls - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        w = torch.where(there, w, torch.zeros_like(w))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        m = lc.amax(1, keepdim=True)
        if score == "sigmoid":
            m = m.clamp(max=0)
        D = torch.where(there, (lc - m).abs(), torch.zeros_like(lc)).amax(1, keepdim=True)
        rel = 2 * (2.0 ** -22 + U * D) + (k + 3) * U
    else:
        w = torch.where(there, s.gather(1, e), torch.zeros((), dtype=torch.float64))
        D = torch.where(there, far.gather(1, e), torch.zeros((), dtype=torch.float64))
        rel = 2.0 ** -22 + U * D + 2 * U
        if score == "softmax":
            rel = rel + 2.0 ** -22 + 1.5 * U * far.amax(1, keepdim=True).clamp(max=20) + (E / 16 + 8) * U
    w = w * scale
    bound = w.abs() * rel * 1.01 + 2.0 ** -125
    w = torch.where(broken[:, None], torch.full_like(w, math.nan), w)
    e = torch.where(there, e, torch.full_like(e, -1))
    flat = e.reshape(-1)
    slots = torch.nonzero(flat >= 0)[:, 0]
    slots = slots[torch.sort(flat[slots], stable=True).indices]
    ends = torch.cumsum(torch.bincount(flat[flat >= 0], minlength=E), 0)
    tokens = torch.full((T * k,), -1, dtype=torch.int64)
    tokens[:len(slots)] = slots // k
    places = torch.full((T * k,), -1, dtype=torch.int64)
    places[slots] = torch.arange(len(slots))
    return w, e, places.view(T, k), ends, tokens, bound


def check_route(r, logits, k, what, **kw):
    w, e, places, ends, tokens, bound = routed(logits, k, **kw)
    for name, got, want in (("experts", r.experts, e), ("ends", r.ends, ends), ("places", r.places, places),
                            ("tokens", r.tokens, tokens)):
        got = got.cpu().long()
        assert got.shape == want.shape, (what, name, got.shape, want.shape)
        if not torch.equal(got, want):
            i = torch.nonzero(got != want)[0].tolist()
            raise AssertionError("%s %s: %d of %d differ, first at %r: %r, want %r" % (
                what, name, int((got != want).sum()), want.numel(), i, got[tuple(i)].item(), want[tuple(i)].item()))
    got = r.weights.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(w)), what + " weights: NaN elsewhere"
    _layer.assert_close(torch.nan_to_num(got), torch.nan_to_num(w), torch.nan_to_num(bound, nan=1.0), what + " weights")


def weights64(l, experts, score, renorm, scale):
    """The weights of chosen experts as a differentiable 64-bit function of the
    logits (choices of -1: 0)."""
    there = experts >= 0
    e = experts.clamp(min=0)
    if score == "softmax":
        s = torch.softmax(l, dim=1).gather(1, e)
    else:
        s = torch.sigmoid(l).gather(1, e)
    s = s * there
    if renorm:
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    return s * scale


def check_route_grad(D, logits, experts, dw, score, renorm, scale, what):
    """D against the formulas, with a bound carried through them."""
    l, e, dw = logits.double().cpu(), experts.long().cpu(), dw.double().cpu()
    T, E = l.shape
    k = e.shape[1]
    there = (e >= 0) & (e < E)
    at = torch.where(there, e, torch.zeros_like(e))
    lc = torch.where(there, l.gather(1, at), torch.full((), -math.inf, dtype=torch.float64))
    dw = torch.where(there, dw, torch.zeros_like(dw))
    top = l.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    far = torch.where(l > -math.inf, top - l, torch.zeros_like(l))
    ones = torch.sigmoid(-lc)  # 1 - s
    if renorm:
        ls = lc if score == "softmax" else torch.nn.functional.logsigmoid(lc)
        m = ls.amax(1, keepdim=True)
        v = torch.exp(ls - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        v = torch.where(there, v, torch.zeros_like(v))
        v = v / v.sum(1, keepdim=True).clamp(min=1e-300)
        D0 = torch.where(there, (lc - lc.amax(1, keepdim=True)).abs(), torch.zeros_like(lc)).amax(1, keepdim=True)
        ev = 2 * (2.0 ** -22 + U * D0) + (k + 3) * U      # relative, of v
        d = (v * dw).sum(1, keepdim=True)
        ed = (v * dw).abs().sum(1, keepdim=True) * (ev + (k + 2) * U)
        g = scale * v * (dw - d)
        eg = abs(scale) * v * ((dw - d).abs() * (ev + 4 * U) + ed + U * (dw.abs() + d.abs()))
        if score == "sigmoid":
            g, eg = g * ones, eg * ones + g.abs() * ones * (2.0 ** -22 + U)
        dense = edense = torch.zeros_like(l)
    elif score == "sigmoid":
        s = torch.where(there, torch.sigmoid(lc), torch.zeros_like(lc))
        g = scale * dw * s * ones
        eg = g.abs() * (2.0 ** -21 + 4 * U)
        dense = edense = torch.zeros_like(l)
    else:
        p = torch.where(l > -math.inf, torch.exp(l - top), torch.zeros_like(l))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        rel = 2.0 ** -21 + U * far + 1.5 * U * far.amax(1, keepdim=True).clamp(max=20) + (E / 16 + 12) * U
        pc = torch.where(there, p.gather(1, at), torch.zeros_like(lc))
        rc = rel.gather(1, at)
        d = (pc * dw).sum(1, keepdim=True)
        ed = ((pc * dw).abs() * (rc + (k + 2) * U)).sum(1, keepdim=True)
        g = scale * pc * dw
        eg = g.abs() * (rc + 3 * U)
        dense = -scale * p * d
        edense = abs(scale) * p * (d.abs() * (rel + 4 * U) + ed)
    want = (dense + torch.zeros_like(l).scatter_add_(1, at, torch.where(there, g, torch.zeros_like(g))))
    bound = edense + torch.zeros_like(l).scatter_add_(1, at, torch.where(there, eg, torch.zeros_like(eg)))
    bound = bound * (1 + k * U) + U * k * want.abs()
    r = torch.finfo(D.dtype).eps / 2 * want.abs() + (2.0 ** -125 if D.dtype == torch.float32 else _layer.TINY[D.dtype])
    _layer.assert_close(D.cpu(), want, (bound * 1.01 + r) * 1.01, what)


# ---- combined rows -----------------------------------------------------------

def rows64(H, places):
    there = (places >= 0) & (places < H.shape[0])
    if H.shape[0] == 0:
        return torch.zeros(places.shape + (H.shape[1],), dtype=torch.float64, device=H.device), there
    r = H.double()[places.long().clamp(0, H.shape[0] - 1)]
    return torch.where(there[:, :, None], r, torch.zeros_like(r)), there


def check_combine(D, H, places, weights, residual, what):
    """k products and additions in FP32, each rounded once against a sum of at
    most S = sum |w h|, the residual's addition, the rounding."""
    r, _ = rows64(H, places)
    k = places.shape[1]
    w = torch.ones(places.shape, dtype=torch.float64, device=H.device) if weights is None else weights.double()
    x = r * w[:, :, None]
    y, S = x.sum(1), x.abs().sum(1)
    e = k * U * S * 1.01
    if residual is not None:
        y = y + residual.double()
        e = e + U * y.abs()
    _layer.assert_close(D, y, (e + _layer.rounding(y, H.dtype)) * 1.01, what)


def check_combine_grad(dh, dw, dY, H, places, weights, before, what):
    """dh: one FP32 product, one rounding, and rows that no place names as they
    were (`before`).  dw: N products summed in FP32 in some order, each addition
    rounded against at most S = sum |dy h|."""
    T, k = places.shape
    R, N = H.shape
    r, there = rows64(H, places)
    dy = dY.double()
    s, S = (r * dy[:, None, :]).sum(2), (r * dy[:, None, :]).abs().sum(2)
    _layer.assert_close(dw, s, S * (N + 16) * U * 1.01 + U * s.abs(), what + " dweights")
    w = torch.ones(places.shape, dtype=torch.float64, device=H.device) if weights is None else weights.double()
    want = before.double().clone()
    bound = torch.zeros_like(want)
    x = (w[:, :, None] * dy[:, None, :])[there]
    at = places[there].long()
    want[at] = x
    bound[at] = (U * x.abs() + _layer.rounding(x, H.dtype)) * 1.01
    _layer.assert_close(dh, want, bound, what + " dh")
