"""fp8_gemm_dgrad_glu and fp8_glu_fwd at infinities and at the ends of the types' ranges: what a call reports
is that of its tensors' own elements, and a derivative that is 0 or 1 is exactly that."""
import pytest
import torch

from tests import glu_reference as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


def cell(v):
    return torch.full((1,), float(v), device="cuda")


def positive(gen, rows, cols, top):
    """FP8 codes of positive finite values: a product of two such tensors has no zero and no NaN."""
    return torch.randint(0x20, top, (rows, cols), generator=gen, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("M,F,N", [(40, 80, 64), (128, 48, 256), (272, 400, 128), (300, 16, 48), (300, 64, 48)])
@pytest.mark.parametrize("act", ["identity", "silu", "gelu"])
def test_an_infinite_gradient_is_an_infinite_maximum(B, M, F, N, act):
    """E5M2 has infinities.  Where F ends inside a 32-column box the kernel multiplies them by the zeros that fill
    it, columns that the tensor does not have."""
    gen = torch.Generator(device="cuda").manual_seed(M + F)
    dy, w = positive(gen, M, N, 0x7B), positive(gen, F, N, 0x60)
    h = torch.rand(M, 2 * F, generator=gen, device="cuda").add_(0.5).to(BF)  # act and act' are not zero there
    dh, q = torch.empty(M, 2 * F, dtype=BF, device="cuda"), torch.empty(M, 2 * F, dtype=torch.uint8, device="cuda")
    amax, sat, scale = cell(7), torch.full((1,), 9, device="cuda"), cell(1e-4)
    kw = dict(act=R.ACTS[act], dh=dh, scale_dh=scale, dh_q=q, amax_out=amax, sat_count=sat)
    B.fp8_gemm_dgrad_glu(dy, w, cell(1), cell(1), h, **kw)
    assert bool(torch.isfinite(dh).all()) and float(amax) == float(dh.abs().max())
    clean = dh.clone()
    dy[7, 3] = 0x7C
    B.fp8_gemm_dgrad_glu(dy, w, cell(1), cell(1), h, **kw)
    others = torch.arange(M, device="cuda") != 7
    assert bool((dh[7] == float("inf")).all()) and torch.equal(dh[others], clean[others])
    assert float(amax) == float("inf")
    codes, count = R.codes_of(dh, scale, torch.float8_e5m2)
    assert torch.equal(q, codes) and int(sat) == count


@pytest.mark.parametrize("M,F,K", [(40, 80, 64), (272, 400, 128), (300, 64, 48)])
def test_scales_whose_product_underflows(B, M, F, K):
    """1 / (s_x s_w) is infinite: so is every element (none of the sums is zero), and the maximum; rows behind M
    and columns behind F, whose sums are zero, count nowhere."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, w, tiny = positive(gen, M, K, 0x60), positive(gen, 2 * F, K, 0x60), cell(1e-20)
    a, amax = torch.empty(M, F, dtype=BF, device="cuda"), cell(7)
    B.fp8_glu_fwd(x, w, tiny, tiny, act=R.ACTS["identity"], act_out=a, amax_out=amax)
    assert bool((a == float("inf")).all()) and float(amax) == float("inf")
    h, dh = torch.ones(M, 2 * F, dtype=BF, device="cuda"), torch.empty(M, 2 * F, dtype=BF, device="cuda")
    B.fp8_gemm_dgrad_glu(x, w[:F], tiny, tiny, h, act=R.ACTS["identity"], dh=dh, amax_out=amax)
    assert bool((dh == float("inf")).all()) and float(amax) == float("inf")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_derivative_far_from_zero_is_one_or_zero(B, act):
    """Finite gates up to BF16's end, past where their squares leave float32: act(g) = g and act'(g) = 1 above,
    0 and 0 below, so the gradient has the bits of the identity's, or is zero."""
    M, F, N = 40, 80, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    dy, w = positive(gen, M, N, 0x30), positive(gen, F, N, 0x30)
    h = torch.randn(M, 2 * F, generator=gen, device="cuda").to(BF)
    far = torch.tensor([1e4, 1e10, 1.8e19, 1.9e19, 1e20, 1e30, 3.38e38], device="cuda")
    g = torch.cat([far, -far]).repeat(6)[:F].to(BF)
    assert bool(torch.isfinite(g).all())
    h[:, :F] = g
    dh, same = torch.empty(M, 2 * F, dtype=BF, device="cuda"), torch.empty(M, 2 * F, dtype=BF, device="cuda")
    amax, scale = cell(0), cell(1e3)
    B.fp8_gemm_dgrad_glu(dy, w, scale, scale, h, act=R.ACTS[act], dh=dh, amax_out=amax)
    B.fp8_gemm_dgrad_glu(dy, w, scale, scale, h, act=R.ACTS["identity"], dh=same)
    up = (g > 0).repeat(2)
    assert bool(torch.isfinite(same).all())
    assert torch.equal(dh[:, up], same[:, up])
    assert bool((dh[:, ~up] == 0).all())
    assert float(amax) == float(dh.abs().max())
