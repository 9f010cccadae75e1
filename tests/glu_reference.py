"""The gated feed-forward block in 64 bits, from its definition, and the tolerances of its GPU tests.

u(T) = half an ulp relative to the value: bf16 2^-8, e4m3 2^-4, e5m2 2^-3; e = 2^-24.
A product's sum of K terms on the tensor core is off by at most 1e-5 sum |a b| (the bound that the
GEMM tests of this suite use).  The activations take an exponential, a reciprocal and under ten
products and sums, each within 2 e, of a z whose own rounding enters as |z| e: 32 e + 2 |z| e of
|act| and of the derivative's terms bound them.  The logistic function sigma = 1 / (1 + 2^t) is 0 where
it lies below float32's normal range, 2^-126 (the reciprocal flushes, and 2^t above 2^126 has no normal
one): so act = g sigma is off by at most |g| 2^-126 there, and the derivative sigma + g sigma (1 - sigma) z'
by (1 + |g z'|) 2^-126.
"""
import math

import torch

E = 2.0 ** -24
UBF = 2.0 ** -8
TINY = 2.0 ** -133  # BF16 subnormals
FLUSH = 2.0 ** -126
ACTS = {"identity": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4}
MAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def act64(name, g):
    """(act, derivative, a bound of |d act / dg| beside which act may be off, |terms| of the derivative)."""
    if name == "identity":
        return g, torch.ones_like(g)
    if name == "relu":
        return g.clamp(min=0), (g > 0).double()
    if name == "relu2":
        return g.clamp(min=0) ** 2, 2 * g.clamp(min=0)
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    th = torch.tanh(z)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def flushed(name, g):
    """What act and its derivative may be off by where the logistic function is flushed."""
    if name not in ("silu", "gelu"):
        return 0.0, 0.0
    slope = 1.0 if name == "silu" else 1.6 + 0.22 * g * g
    return g.abs() * FLUSH, (1 + g.abs() * slope) * FLUSH


def z_of(name, g):
    """|argument of the exponential|."""
    if name == "silu":
        return g.abs()
    if name == "gelu":
        return 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3).abs()
    return torch.zeros_like(g)


def rounded(v, tol):
    """Allowed error of BF16(v~) with |v~ - v| <= tol."""
    return tol + UBF * (v.abs() + tol) + TINY


def fwd(x, w, name):
    """(g, u, a, tolerances of BF16 g, u, a) for float64 operands x [M,K], w [2F,K] (scales applied)."""
    F = w.shape[0] // 2
    h, size = x @ w.T, x.abs() @ w.abs().T
    th = 1e-5 * size + 4 * E * h.abs()
    g, u = h[:, :F], h[:, F:]
    tg, tu = th[:, :F], th[:, F:]
    f, d = act64(name, g)
    # |act(g~) - act(g)| <= max |act'| tg: the derivative moves by at most 2 tg (ReLU^2, the others' second
    # derivatives are below 2) on the way
    tf = (d.abs() + 2 * tg) * tg + (32 + 2 * z_of(name, g)) * E * f.abs() + flushed(name, g)[0]
    ta = (f.abs() + tf) * tu + u.abs() * tf + 2 * E * (f * u).abs()
    return g, u, f * u, rounded(g, tg), rounded(u, tu), rounded(f * u, ta)


def bwd(dy, w2, h, name):
    """(dh, tolerance) for float64 dy [M,N], w2 [F,N] (scales applied) and h [M,2F]."""
    F = w2.shape[0]
    dA, size = dy @ w2.T, dy.abs() @ w2.abs().T
    tA = 1e-5 * size + 4 * E * dA.abs()
    g, u = h[:, :F], h[:, F:]
    f, d = act64(name, g)
    rel = (32 + 2 * z_of(name, g)) * E
    # the derivative's terms: sigma <= 1 and f (1 - sigma) z'; |z'| <= 1.6 + 0.22 g^2 (GELU), and f (1 - sigma)
    # z' is below 1.2 wherever it is not in the exponential's tail
    td = rel * (d.abs() + 1.2) if name in ("silu", "gelu") else rel * d.abs()
    ff, fd = flushed(name, g)
    td, tf = td + fd, rel * f.abs() + ff
    dg, du = dA * u * d, dA * f
    tg = (tA * (d.abs() + td) + dA.abs() * td) * u.abs() + 3 * E * dg.abs()
    tu = tA * (f.abs() + tf) + dA.abs() * tf + 3 * E * du.abs()
    v, t = torch.cat([dg, du], 1), torch.cat([tg, tu], 1)
    return v, rounded(v, t)


def assert_within(got, want, tol, name):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside tolerance; first at {i}: got {float(got[i])!r}, "
                             f"want {float(want[i])!r}, tolerance {float(tol[i]):.3e}")


def codes_of(v, scale, fmt):
    """FP8 codes (bytes) of BF16 values under a float32 scale, and the saturation count."""
    s = v.float() * scale
    return s.clamp(-MAX[fmt], MAX[fmt]).to(fmt).view(torch.uint8), int((s.abs() > MAX[fmt]).sum())
