"""block_norm_bwd of rows that the CTAs of a cluster share, with every number of sums that a row can have: two
(a norm before the next block, and one after this one or a gate's gradient), one, or none, and dalpha beside them."""
import pytest
import torch

from tests.test_block_norm_gpu import BF, EPS, FP, HF, check_bwd, make

pytestmark = pytest.mark.gpu

# two, two, four and eight CTAs a row; on and off the 16-byte grid
WIDE = [(12288, BF), (8200, HF), (16377, BF), (6000, FP), (9001, FP), (40000, BF)]


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("M", [1, 4, 231])
@pytest.mark.parametrize("N,T", WIDE)
@pytest.mark.parametrize("alpha", [False, True])
def test_parts_over_a_cluster(B, N, T, M, alpha):
    """A cluster's rows are an odd count at 1 and 4 (one each), and odd in some and even in others at 231."""
    for pre, post, block, gate in ((1, 0, 1, 0), (1, 0, 0, 0), (1, 1, 1, 0), (1, 0, 1, 1), (0, 0, 1, 0), (0, 1, 1, 1), (0, 0, 0, 0)):
        check_bwd(B, M, N, T, pre=bool(pre), post=bool(post), block=bool(block), gate=bool(gate), alpha=alpha)


@pytest.mark.parametrize("N,T", [(12288, BF), (16377, HF), (6000, FP), (40000, BF)])
@pytest.mark.parametrize("block", [False, True])
def test_one_sum_a_row_repeats(B, N, T, block):
    """The same bits from call to call where the last row's sum is all that the CTAs exchange before dalpha."""
    M = 231
    s = make(M, N, T, 8, alpha=True)
    rstd = (s["r"].float().square().mean(1) + EPS).rsqrt()
    ws = torch.empty(B.block_norm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(20):
        out = dict(dresidual=torch.empty_like(s["r"]), dweight=torch.empty(N, device="cuda"), dalpha=torch.empty(1, device="cuda"))
        if block:
            out |= dict(dx=torch.empty_like(s["r"]), dpost_weight=torch.empty(N, device="cuda"))
        B.block_norm_bwd(s["dy"], s["r"], rstd, s["w"], dr=s["dr"], x=s["x"] if block else None, residual=s["residual"],
                         alpha=s["alpha"], post_weight=s["wp"], workspace=ws, **out)
        first = first or out
        assert all(torch.equal(out[k], first[k]) for k in out)
