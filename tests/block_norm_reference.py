"""block_norm_fwd and its gradient in 64 bits, from their definitions, and the tolerances of their tests.

u(T) = half an ulp of the type: 2^-8 (bfloat16), 2^-11 (float16), 2^-24 (float32); e = 2^-24.  A
float32 sum whose longest chain has L additions is off by at most L e sum |terms|: a thread adds at
most 64 terms of a row, or N / 512 where rows are wider than the one-pass kernels take, and at most
5 + 16 joins follow: L(N) = 64 + N / 256 + 32.  A column sum is bounded by M + 32 additions, the sum of
all elements by 16 M + N + 64 (a thread's 16 columns of at most M rows).  Each elementwise step adds e.
"""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E = 2.0 ** -24


def chain(N):
    return 64 + N // 256 + 32


def rounded(v, tol, T):
    return tol + U[T] * (v.abs() + tol) + TINY[T]


def stream(x, residual, wp, gate, alpha, post, eps):
    """(r before rounding, rstd_post, tolerance of the float32 r, of rstd_post)."""
    N = x.shape[1]
    rp = (x.square().mean(1) + eps).rsqrt() if post else torch.ones_like(x[:, 0])
    rel = (chain(N) + 2) * E / 2 + 4 * E if post else 0.0
    b = x * rp[:, None] * wp * gate[:, None]
    r = b + (alpha * residual if residual is not None else 0.0)
    size = b.abs() + ((alpha * residual).abs() if residual is not None else 0.0)
    return r, rp, b.abs() * rel + 6 * E * size, rel * rp


def norm(r, w, eps):
    """(y, rstd, tolerance of the float32 y, of rstd) of the stored r."""
    rstd = (r.square().mean(1) + eps).rsqrt()
    rel = (chain(r.shape[1]) + 2) * E / 2 + 4 * E
    y = r * rstd[:, None] * w
    return y, rstd, y.abs() * (rel + 4 * E), rel * rstd


def bwd(dy, r, rstd, w, dr_in, x, rp, wp, gate, alpha, residual, post):
    """{name: (value, tolerance before a rounding to T)}; dy None: no norm before a next block."""
    M, N = x.shape
    L, Lc = chain(N), M + 32
    out = {}
    dr = dr_in if dr_in is not None else torch.zeros_like(x)
    t = E * dr.abs()
    if dy is not None:
        rhat, g = r * rstd[:, None], dy * w
        c = (g * rhat).mean(1, keepdim=True)
        tc = (L + 6) * E * (g * rhat).abs().mean(1, keepdim=True)
        out["dweight"] = (dy * rhat).sum(0), (Lc + 4) * E * (dy * rhat).abs().sum(0)
        t = rstd[:, None] * (rhat.abs() * tc + 6 * E * (g.abs() + (rhat * c).abs())) + 2 * t
        dr = dr + rstd[:, None] * (g - rhat * c)
        t = t + 2 * E * dr.abs()
    out["dresidual"] = alpha * dr, abs(alpha) * (t + E * dr.abs())
    if residual is not None:
        out["dalpha"] = ((dr * residual).sum().reshape(1),
                         ((t * residual.abs()).sum() + (16 * M + N + 64) * E * (dr * residual).abs().sum()).reshape(1))
    xhat = x * rp[:, None] if post else x
    v = dr * gate[:, None] * xhat
    out["dpost_weight"] = v.sum(0), (Lc + 6) * E * v.abs().sum(0) + (t * gate[:, None].abs() * xhat.abs()).sum(0)
    d = dr * wp
    e = (d * xhat).sum(1, keepdim=True)
    te = (t * (wp * xhat).abs()).sum(1, keepdim=True) + (L + 6) * E * (d * xhat).abs().sum(1, keepdim=True)
    out["dgate"] = e[:, 0], te[:, 0]
    k = gate[:, None] * (rp[:, None] if post else 1.0)
    if post:
        dx = k * (d - xhat * e / N)
        tx = k.abs() * (t * wp.abs() + xhat.abs() * te / N + 6 * E * (d.abs() + (xhat * e / N).abs())) + 3 * E * dx.abs()
    else:
        dx = k * d
        tx = k.abs() * t * wp.abs() + 3 * E * dx.abs()
    out["dx"] = dx, tx
    return out


def assert_within(got, want, tol, name):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside tolerance; first at {i}: got {float(got[i])!r}, "
                             f"want {float(want[i])!r}, tolerance {float(tol[i]):.3e}")
