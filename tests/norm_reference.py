"""Layer norm, its gradient and dropout in 64 bits, from their definitions (numpy and
torch on the CPU; nothing of the CUDA library), and the tolerances of the GPU tests.

Tolerances.  u(T) = half an ulp of the output type: 2^-8 (bfloat16), 2^-11 (float16),
2^-24 (float32); e = 2^-24.  A float32 sum whose longest chain has L additions is off by
at most L e sum |terms|.  In the kernels a thread adds at most 64 terms of a row in a
chain (or N / 1024 quads where a row is wider than 64 terms a thread), and 5 + 5 shuffles
follow, so L(N) = 64 + N / 256 + 16 covers a row sum; a column sum is bounded by L = M + 16
whatever the split of the rows.  Each elementwise step adds e.
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half the smallest spacing: what a subnormal result may be off by
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E = 2.0 ** -24


def row_chain(N):
    return 64 + N // 256 + 16


def philox(ctr, key):
    """Philox4x32-10 of uint32 counter words (c0, c1, c2, c3) and key words (k0, k1); arrays broadcast."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in ctr]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(seed, offset, M, N, p, row0=0):
    """The keep mask [M, N] of rows row0 .. row0 + M."""
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    quads = -(-N // 4)
    words = philox((np.arange(quads)[None, :], np.arange(row0, row0 + M)[:, None], offset & 0xFFFFFFFF, offset >> 32),
                   (seed & 0xFFFFFFFF, seed >> 32))
    w = np.stack([np.broadcast_to(v, (M, quads)) for v in words], axis=2).reshape(M, 4 * quads)[:, :N]
    return w >= np.uint64(round(p * 2 ** 32))


def residual_stream(x, residual, keep, p):
    """r = T(float32(residual + (keep ? float32(x * inv) : 0))), bit for bit: CPU float32 operations on CPU tensors."""
    v = x.float()
    if keep is not None:
        inv = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
        v = torch.where(torch.from_numpy(keep), v * torch.tensor(inv), torch.zeros(()))
    if residual is not None:
        v = residual.float() + v
    return v.to(x.dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def norm_fwd(r, w, b, eps):
    """(y, mean, rstd) in float64 of the float64 rows r."""
    mean = r.mean(1)
    d = r - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + b, mean, rstd


def fwd_tolerances(r, w, b, eps, T):
    """Allowed |error| of (y, mean, rstd) for float64 rows r."""
    N = r.shape[1]
    L = row_chain(N)
    y, mean, rstd = norm_fwd(r, w, b, eps)
    d = r - mean[:, None]
    t_mean = (L + 2) * E * np.abs(r).mean(1)
    # the variance: its own sum, the rounding of each deviation, and the mean's error, which enters
    # squared (the deviations from the exact mean sum to zero) -- relative to var + eps
    rel_var = (L + 6) * E + t_mean ** 2 * rstd ** 2 + 2 * E * np.abs(d).mean(1) * np.abs(r).max(1) * rstd ** 2
    t_rstd = rstd * (0.5 * rel_var / np.maximum(1 - rel_var, 0.5) + 4 * E)
    t_y = (np.abs(w) * (rstd[:, None] * (t_mean[:, None] + 2 * E * np.abs(d)) + np.abs(d) * t_rstd[:, None] * 1.01)
           + 4 * E * (np.abs(d * rstd[:, None] * w) + np.abs(b)))
    return t_y + U[T] * (np.abs(y) + t_y) + TINY[T], t_mean, t_rstd


def norm_bwd(dy, r, mean, rstd, w, dres):
    """(dr, dweight, dbias) in float64."""
    xhat = (r - mean[:, None]) * rstd[:, None]
    g = dy * w
    dr = rstd[:, None] * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    if dres is not None:
        dr = dr + dres
    return dr, (dy * xhat).sum(0), dy.sum(0)


def bwd_tolerances(dy, r, mean, rstd, w, dres, T, inv=1.0):
    """Allowed |error| of (dx, dbranch, dweight, dbias); mean and rstd are the float32 values given."""
    M, N = dy.shape
    L = row_chain(N)
    xhat = (r - mean[:, None]) * rstd[:, None]
    t_xhat = E * (np.abs(r) + np.abs(mean)[:, None]) * rstd[:, None] + 2 * E * np.abs(xhat)  # difference, product
    g = dy * w
    dr, _, _ = norm_bwd(dy, r, mean, rstd, w, dres)
    c2 = np.abs((g * xhat).mean(1, keepdims=True))
    t_c1 = (L + 4) * E * np.abs(g).mean(1, keepdims=True)
    t_c2 = (L + 5) * E * np.abs(g * xhat).mean(1, keepdims=True) + (np.abs(g) * t_xhat).mean(1, keepdims=True)
    size = np.abs(g) + np.abs(g.mean(1, keepdims=True)) + np.abs(xhat) * c2
    t = rstd[:, None] * (t_c1 + (np.abs(xhat) + t_xhat) * t_c2 + t_xhat * c2 + 6 * E * size)
    if dres is not None:
        t = t + 2 * E * (np.abs(dr) + np.abs(dres))
    t_dx = t + U[T] * (np.abs(dr) + t) + TINY[T]
    t_db = inv * t + (U[T] + 2 * E) * inv * (np.abs(dr) + t) + TINY[T]
    Lc = M + 16
    t_dw = (Lc + 3) * E * np.abs(dy * xhat).sum(0) + (np.abs(dy) * t_xhat).sum(0)
    t_dbias = Lc * E * np.abs(dy).sum(0)
    return t_dx, t_db, t_dw, t_dbias


def assert_within(got, want, tol, name):
    err = np.abs(np.asarray(got, dtype=np.float64) - want)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside tolerance; first at {i}: got "
                             f"{np.asarray(got)[i]!r}, want {want[i]!r}, tolerance {np.broadcast_to(tol, want.shape)[i]:.3e}")
