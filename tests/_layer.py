"""References and error bounds for the layer products' tests: 64-bit plain
forms on the CPU or GPU, sharing no code with the library.

Bounds.  u = 2^-24 is half a step of FP32, h = eps / 2 half a step of the
output type.
* P, a sum of K products in FP32, in any order: the products of two 16-bit
  values are exact in FP32, each of at most K additions rounds by u relative
  to a partial sum of at most S = sum |a b|: |P' - P| <= K u S (1 + K u).
* Z = P + bias: one more rounding, u |Z|.
* act(z): its slope is at most 1.13 in size (GELU), so an error e of z gives
  1.13 e.  Evaluating it: z times a value in [0, 1] that comes from one
  exponential, one reciprocal (each within 2^-22 of its value), a polynomial
  (2^-19 of its value) and an exponent's argument w rounded by 2^-23 |w|;
  where |w| > 104 the exponential, and so the value or its distance from 1,
  is below 2^-149, so its relative error is below 104 2^-22 + 2^-18 < 2^-15.
  A value of the form 1 - q keeps an absolute error of 2^-22 on top.
  So: 2^-15 |act(z)| + 2^-22 |z|.
* act'(z) = s + z r, with the same kind of error in both terms: 2^-15 (|s| +
  |z r|) + 2^-21.
* residual: one rounding, u |D|.  The final rounding: h |D| plus half the
  smallest subnormal.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
GEN = {"f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def act64(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    """act'(z) and the sum of the sizes of its terms."""
    if act == "relu":
        s = (z > 0).double()
        return s, torch.zeros_like(s)
    if act == "gelu":
        F = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        t = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        # (0.5 (1 + tanh u) as a logistic: it keeps its precision in the tail)
        F = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        t = z * F * (1 - F) * 2 * c * (1 + 3 * 0.044715 * z * z)
    else:
        F = torch.sigmoid(z)
        t = z * F * (1 - F)
    return F + t, F.abs() + t.abs()


def product64(A, B, layout):
    """P and S = sum |a b| in 64 bits (on the operands' device)."""
    a, b = A.double(), B.double()
    if layout == "nt":
        b = b.t().contiguous()
    elif layout == "tn":
        a = a.t().contiguous()
    return a @ b, a.abs() @ b.abs()


def rounding(d, dt):
    return torch.finfo(dt).eps / 2 * d.abs() + TINY[dt]


def assert_close(got, want, bound, what):
    g = got.double()
    err = (g - want).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err - bound, torch.full_like(err, -1.0))))
        w = want.expand_as(g).reshape(-1)[i]
        raise AssertionError("%s: %d of %d off; worst at %d: got %r, want %r, bound %r" % (
            what, int(bad.sum()), g.numel(), i, g.reshape(-1)[i].item(), w.item(),
            bound.expand_as(g).reshape(-1)[i].item()))


def check_forward(D, Z, A, B, layout, bias, act, residual, what):
    """D (and Z, unless None) against the forward epilogue of A, B."""
    K = A.shape[1]
    P, S = product64(A, B, layout)
    eP = K * U * S * 1.01
    z = P if bias is None else P + bias.double()
    eZ = eP + U * z.abs()
    if Z is not None:
        assert_close(Z, z, (eZ + rounding(z, A.dtype)) * 1.01, what + " Z")
    d = act64(z, act)
    e = eZ if act == "none" else 1.13 * eZ + 2.0 ** -15 * d.abs() + 2.0 ** -22 * z.abs()
    if residual is not None:
        d = d + residual.double()
        e = e + U * d.abs()
    assert_close(D, d, (e + rounding(d, A.dtype)) * 1.01, what + " D")


def check_dact(D, A, B, layout, Z, act, what):
    K = A.shape[1]
    P, S = product64(A, B, layout)
    s, mag = slope64(Z.double(), act)
    d = P * s
    e = K * U * S * 1.01 * s.abs() + P.abs() * (2.0 ** -15 * mag + 2.0 ** -21) + U * d.abs()
    assert_close(D, d, (e + rounding(d, A.dtype)) * 1.01, what)


def check_tn(D, c, A, B, what):
    K = A.shape[0]
    P, S = product64(A, B, "tn")
    assert_close(D, P, (K * U * S * 1.01 + rounding(P, A.dtype)) * 1.01, what + " D")
    if c is not None:
        s, m = A.double().sum(0), A.double().abs().sum(0)
        assert_close(c, s, (K * U * m * 1.01 + rounding(s, A.dtype)) * 1.01, what + " colsum")


def spans(ends):
    lo = 0
    for g, e in enumerate(ends):
        yield g, lo, e
        lo = e
