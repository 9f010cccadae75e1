"""Outputs of the block norms over their inputs where a row's lanes do not wait for one another: calls without a
norm, whose warps (or CTAs) run ahead of each other by rows, on and off the 16-byte grid, and rows of every kernel."""
import pytest
import torch

from tests.test_block_norm_gpu import BF, EPS, FP, HF, make

pytestmark = pytest.mark.gpu

SIZES = [(700, 200, BF), (700, 203, HF), (300, 1601, BF), (300, 5000, BF), (300, 5001, HF), (120, 12288, BF), (120, 16377, HF), (120, 9001, FP),
         (40, 20001, BF), (12, 70001, BF), (12, 40002, FP)]


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("M,N,T", SIZES)
@pytest.mark.parametrize("post,pre", [(False, False), (True, False), (False, True)])
def test_forward(B, M, N, T, post, pre):
    s = make(M, N, T, N, gate=True, alpha=True)
    r, y = torch.empty_like(s["x"]), torch.empty_like(s["x"]) if pre else None
    kw = dict(eps=EPS, alpha=s["alpha"], gate=s["gate"], post_weight=s["wp"], post_norm=post)
    w = s["w"] if pre else None
    B.block_norm_fwd(s["x"], w, y, residual=s["residual"], r_out=r, **kw)
    for over in ("x", "residual"):
        x, residual = s["x"].clone(), s["residual"].clone()
        first, second = (x, residual) if over == "x" else (residual, x)
        B.block_norm_fwd(x, w, second if pre else None, residual=residual, r_out=first, **kw)
        assert torch.equal(first, r) and (not pre or torch.equal(second, y)), over


@pytest.mark.parametrize("M,N,T", SIZES)
@pytest.mark.parametrize("post,pre", [(False, False), (True, False), (False, True)])
def test_backward(B, M, N, T, post, pre):
    s = make(M, N, T, N, alpha=True)
    rstd = (s["r"].float().square().mean(1) + EPS).rsqrt() if pre else None
    rp = (s["x"].float().square().mean(1) + EPS).rsqrt() if post else None
    ws = torch.empty(B.block_norm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")

    def call(t, dresidual, dx):
        sums = dict(dpost_weight=torch.empty(N, device="cuda"), dalpha=torch.empty(1, device="cuda"))
        B.block_norm_bwd(t["dy"] if pre else None, t["r"] if pre else None, rstd, s["w"] if pre else None, dr=t["dr"], x=t["x"],
                         residual=t["residual"], alpha=s["alpha"], post_weight=s["wp"], post_norm=post, rstd_post=rp, dresidual=dresidual,
                         dx=dx, workspace=ws, **sums)
        return [dresidual, dx, *sums.values()]

    want = call(s, torch.empty_like(s["x"]), torch.empty_like(s["x"]))
    for a, b in (("dr", "x"), ("residual", "dr"), ("x", "residual")) + ((("dy", "r"),) if pre else ()):
        t = {k: s[k].clone() for k in ("dy", "r", "dr", "x", "residual")}
        got = call(t, t[a], t[b])
        assert all(torch.equal(g, v) for g, v in zip(got, want)), (a, b)
