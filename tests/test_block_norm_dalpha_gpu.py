"""dalpha where it does not cancel: residual is the gradient that it meets, so dalpha = sum dr'^2, and a bound by
the length of the float32 chains is a small part of it: a row, a CTA or a cluster that were left out would show.

Chain: half of a pair of a lane's at most 32 columns, 16 additions a row, M rows at most; then one join of the
pair, 5 of the warp, at most 128 of a cluster's warps, and of at most 1024 partial sums 2 a thread, 5 and 16 more:
16 M + 160.  (The reference's own bound, 16 M + N + 64, also covers rows wider than clusters take.)"""
import pytest
import torch

from tests import block_norm_reference as R
from tests.test_block_norm_gpu import BF, EPS, FP, HF, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("M", [1, 37, 400])
@pytest.mark.parametrize("N,T", [(64, BF), (203, HF), (768, BF), (1001, FP), (1600, BF), (1601, BF), (5000, BF), (8192, BF), (8200, HF),
                                 (12288, BF), (16377, HF), (6000, FP), (9001, FP), (40000, BF)])
@pytest.mark.parametrize("post,block", [(True, True), (False, True), (False, False)])
def test_dalpha_that_does_not_cancel(B, M, N, T, post, block):
    s = make(M, N, T, M + N, gate=True, alpha=True)
    rstd = (s["r"].float().square().mean(1) + EPS).rsqrt()
    rp = (s["x"].float().square().mean(1) + EPS).rsqrt() if post else None

    def want(residual):
        return R.bwd(f64(s["dy"]), f64(s["r"]), f64(rstd), f64(s["w"]), f64(s["dr"]), f64(s["x"]), f64(rp), f64(s["wp"]), f64(s["gate"]),
                     1.0, residual, post)

    dr, t = want(None)["dresidual"]  # alpha 1: dr' and the bound of its own error
    residual = dr.to(T)
    value = (dr * f64(residual)).sum()
    tol = (t * f64(residual).abs()).sum() + (16 * M + 160) * R.E * (dr * f64(residual)).abs().sum()
    assert float(tol) < 1e-3 * float(value)
    dalpha = torch.full((1,), 7.0, device="cuda")
    out = dict(dx=torch.empty_like(residual), dgate=torch.empty(M, device="cuda")) if block and post else dict(dx=torch.empty_like(residual)) if block else {}
    ws = torch.full((B.block_norm_bwd_workspace_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")
    B.block_norm_bwd(s["dy"], s["r"], rstd, s["w"], dr=s["dr"], x=s["x"] if block else None, residual=residual, alpha=s["alpha"],
                     gate=s["gate"], post_weight=s["wp"], post_norm=post, rstd_post=rp, dalpha=dalpha, workspace=ws, **out)
    R.assert_within(dalpha, value.reshape(1), tol.reshape(1), "dalpha")
