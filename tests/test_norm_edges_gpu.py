"""The layer norm's gradient at the edges of its range on the GPU: rows whose mean is far above
their deviation, and rows so narrow in value that the square of rstd passes float32 (eps = 0).

Tolerances (e = 2^-24, L the longest chain of a row's sum, norm_reference.row_chain).  mean and
rstd are inputs, so xhat = (r - mean) rstd costs one rounding of the difference and one of the
product, each relative to itself: 2 e |xhat|, however far the mean.  Then
    c1 = sum g / N         (L + 4) e mean |g|          a sum, two roundings of the division, g's own
    c2 = sum g xhat / N    (L + 7) e mean |g xhat|     the same and xhat's
    g - c1 - xhat c2       3 e |xhat c2| + 2 e (|g| + |c1| + |xhat c2|)
    times rstd, + dres     2 e (|dr| + |dres|)
and the output's own rounding.  The column sums: the chain of rows, xhat's two roundings and the
product's."""
import numpy as np
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from tests import norm_reference as R
from tests.norm_reference import E, assert_within, f64
from tests.test_norm_gpu import BF, SF, ids, params, rng_of, rows, run_bwd, stats

pytestmark = pytest.mark.gpu


def tolerances(dy, r, mean, rstd, w, dres, T, inv):
    """Allowed |error| of (dx, dbranch, dweight, dbias) for float64 inputs."""
    M, N = dy.shape
    L = R.row_chain(N)
    xhat = (r - mean[:, None]) * rstd[:, None]
    g = dy * w
    c1, c2 = np.abs(g.mean(1, keepdims=True)), np.abs((g * xhat).mean(1, keepdims=True))
    dr = R.norm_bwd(dy, r, mean, rstd, w, dres)[0]
    t_c1, t_c2 = (L + 4) * E * np.abs(g).mean(1, keepdims=True), (L + 7) * E * np.abs(g * xhat).mean(1, keepdims=True)
    size = np.abs(g) + c1 + np.abs(xhat) * c2
    t = rstd[:, None] * (t_c1 + np.abs(xhat) * t_c2 + 3 * E * np.abs(xhat) * c2 + 2 * E * size)
    t = t + 2 * E * (np.abs(dr) + (0.0 if dres is None else np.abs(dres)))
    t_dx = t + R.U[T] * (np.abs(dr) + t) + R.TINY[T]
    t_db = inv * t + (R.U[T] + 2 * E) * inv * (np.abs(dr) + t) + R.TINY[T]
    chain = M + 16
    return t_dx, t_db, (chain + 4) * E * np.abs(dy * xhat).sum(0), chain * E * np.abs(dy).sum(0)


def check(dy, r, w, eps, dres=None, p=0.0):
    M, N = dy.shape
    T = dy.dtype
    mean, rstd = stats(r, eps)
    assert bool(rstd.isfinite().all())
    dx, db, dweight, dbias = run_bwd(dy, r, mean, rstd, w, dres=dres, p=p, rng=rng_of(1, 2), want_branch=True)
    args = (f64(dy), f64(r), f64(mean), f64(rstd), f64(w), None if dres is None else f64(dres))
    dr, dw, dbs = R.norm_bwd(*args)
    inv = 1.0 / (1.0 - p)
    t_dx, t_db, t_dw, t_dbias = tolerances(*args, T, inv)
    keep = R.keep_mask(1, 2, M, N, p)
    assert_within(f64(dx), dr, t_dx, "dx")
    assert_within(f64(db), np.where(keep, dr * inv, 0.0), t_db, "dbranch")
    assert_within(f64(dweight), dw, t_dw, "dweight")
    assert_within(f64(dbias), dbs, t_dbias, "dbias")


# every kernel: lanes, one warp, two and more warps, a whole CTA a row, the loop over wide rows; on and off the grid
WIDTHS = [5, 64, 768, 1001, 1600, 2056, 4099, 6400, 12345, 16384, 20000]


def with_xhat_part(r, N, T, seed, eps):
    """A dy that has a part along xhat, so that c2 is of the size of g."""
    mean, rstd = stats(r, eps)
    xhat = (r.double() - mean.double()[:, None]) * rstd.double()[:, None]
    return (rows(r.shape[0], N, SF, seed).double() + 0.5 * xhat).to(T)


@pytest.mark.parametrize("mean,std", [(1e3, 1.0), (-1e5, 1.0), (1e3, 1e-2)])
@pytest.mark.parametrize("N", WIDTHS)
def test_bwd_of_a_far_mean(N, mean, std):
    M = 13
    r = rows(M, N, SF, 101, std=std, mean=mean)
    w, _ = params(N, SF, 102)
    dy = with_xhat_part(r, N, SF, 103, 1e-5)
    check(dy, r, w, 1e-5)
    check(dy, r, w, 1e-5, dres=rows(M, N, SF, 104), p=0.2)


@pytest.mark.parametrize("T", [BF, SF], ids=ids.get)
@pytest.mark.parametrize("N", WIDTHS)
def test_bwd_of_a_tiny_deviation_without_eps(N, T):
    """rstd = 1e20 is finite, its square is not."""
    M = 13
    r = rows(M, N, T, 111, std=1e-20)
    w, _ = params(N, SF, 112)
    dy = with_xhat_part(r, N, T, 113, 0.0)
    check(dy, r, w, 0.0)
    check(dy, r, w, 0.0, dres=rows(M, N, T, 114, std=1e20), p=0.2)
