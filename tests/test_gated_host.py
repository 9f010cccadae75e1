"""The gated block's calls and the norms before and after a block without a GPU: the tests' references
against autograd and differences, the argument checks of the C entry points, of the binding and of
Fp8GatedMlpStack.  No kernel is launched; the pointers passed here are never dereferenced."""
import ctypes

import pytest
import torch

from tests import block_norm_reference as RN
from tests import glu_reference as RG
from quantize_fp8_gemm_gb300 import binding as B
from quantize_fp8_gemm_gb300.gatedstack import Fp8GatedMlpStack

OK, ERR_NULL, ERR_ALIGN, ERR_SHAPE, ERR_UNSUPPORTED, ERR_CUDA = range(6)
A = 1 << 20  # an aligned fake device address
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would launch on the fake addresses")


@pytest.fixture(scope="module")
def lib():
    from quantize_fp8_gemm_gb300 import build
    build.build()
    return B.lib()


@pytest.mark.parametrize("act", list(RG.ACTS))
def test_gated_reference_against_differences(act):
    torch.manual_seed(1)
    dy, w2, h = torch.randn(5, 7, dtype=torch.float64), torch.randn(6, 7, dtype=torch.float64), torch.randn(5, 12, dtype=torch.float64)

    def loss(h):
        return ((RG.act64(act, h[:, :6])[0] * h[:, 6:]) @ w2 * dy).sum()

    dh, _ = RG.bwd(dy, w2, h, act)
    for i in range(5):
        for j in range(12):
            d = torch.zeros_like(h)
            d[i, j] = 1e-6
            assert abs((loss(h + d) - loss(h - d)) / 2e-6 - dh[i, j]) < 1e-6 * (1 + dh[i, j].abs())
    fn = dict(silu=torch.nn.functional.silu, gelu=lambda v: torch.nn.functional.gelu(v, approximate="tanh"), relu=torch.relu,
              relu2=lambda v: torch.relu(v) ** 2, identity=lambda v: v)[act]
    x, w = torch.randn(4, 9, dtype=torch.float64), torch.randn(10, 9, dtype=torch.float64)
    a = RG.fwd(x, w, act)[2]
    assert torch.allclose(a, fn(x @ w[:5].T) * (x @ w[5:].T), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_norm_reference_against_autograd(post, pre):
    torch.manual_seed(2)
    r = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    x, res, wp, w, gate, alpha = r(5, 33), r(5, 33), r(33), r(33), r(5), torch.tensor(0.7, dtype=torch.float64)
    leaves = [t.requires_grad_() for t in (x, res, wp, w, gate, alpha)]
    dy, dr = r(5, 33), r(5, 33)
    eps = 1e-5
    s, rp, *_ = RN.stream(x, res, wp, gate, alpha, post, eps)
    y, rstd, *_ = RN.norm(s, w, eps)
    ((s * dr).sum() + ((y * dy).sum() if pre else 0.0)).backward()
    with torch.no_grad():
        got = RN.bwd(dy if pre else None, s.detach(), rstd.detach(), w, dr, x, rp.detach(), wp, gate, float(alpha), res, post)
    want = dict(dx=x.grad, dresidual=res.grad, dpost_weight=wp.grad, dgate=gate.grad, dalpha=alpha.grad.reshape(1))
    if pre:
        want["dweight"] = w.grad
    for name, v in want.items():
        assert torch.allclose(got[name][0], v, rtol=1e-10, atol=1e-11), name
    assert len(leaves) == 6


def glu(lib, x=A, w=A, sx=A, sw=A, act=3, h=A, a=A, s=A, q=A, qt=A, amax=A, sat=A, M=32, F=48, K=64, flags=0, st=None):
    args = B.GluArgs(x, w, sx, sw, h, a, s, q, qt, amax, sat, M, F, K, act, flags, st)
    return lib.fp8_glu_fwd(ctypes.byref(args), None)


def dglu(lib, dy=A, w=A, sdy=A, sw=A, h=A, act=3, dh=A, s=A, q=A, qt=A, amax=A, sat=A, M=32, N=64, F=48, flags=0, st=None):
    args = B.DgradGluArgs(dy, w, sdy, sw, h, dh, s, q, qt, amax, sat, M, N, F, act, flags, st)
    return lib.fp8_gemm_dgrad_glu(ctypes.byref(args), None)


def test_gated_argument_checks(lib):
    assert lib.fp8_glu_fwd(None, None) == ERR_NULL and lib.fp8_gemm_dgrad_glu(None, None) == ERR_NULL
    for call, width in ((glu, "K"), (dglu, "N")):
        for k in ("w", "sw", "s"):
            assert call(lib, **{k: None}) == ERR_NULL, k
        for act in (-1, 5):
            assert call(lib, act=act) == ERR_UNSUPPORTED
        assert call(lib, flags=2) == ERR_UNSUPPORTED
        assert call(lib, M=-1) == ERR_SHAPE and call(lib, M=1 << 31, qt=None) == ERR_SHAPE
        for k in ("F", width):
            for bad in (0, 8, 24, 1 << 31):
                assert call(lib, **{k: bad}) == ERR_SHAPE, (k, bad)
        assert call(lib, M=33) == ERR_SHAPE  # transposed codes of rows that are no 16-byte multiple
        for k in ("w", "h", "q", "qt"):
            assert call(lib, **{k: A + 8}) == ERR_ALIGN, k
        assert call(lib, s=A + 2) == ERR_ALIGN and call(lib, sat=A + 4) == ERR_ALIGN and call(lib, st=A + 1) == ERR_ALIGN
    assert glu(lib, x=None) == ERR_NULL and glu(lib, sx=None) == ERR_NULL and glu(lib, a=A + 8) == ERR_ALIGN
    assert glu(lib, a=None, q=None, qt=None) == ERR_NULL
    assert dglu(lib, dy=None) == ERR_NULL and dglu(lib, h=None) == ERR_NULL and dglu(lib, dh=A + 8) == ERR_ALIGN
    assert dglu(lib, dh=None, q=None, qt=None) == ERR_NULL


@no_gpu
def test_gated_well_formed(lib):
    """Only the device check remains, and there is no sm_103 here."""
    for call in (glu, dglu):
        for kw in ({}, dict(q=None, qt=None, s=None, sat=None), dict(M=33, qt=None), dict(amax=None, sat=None), dict(act=4)):
            assert call(lib, **kw) == ERR_UNSUPPORTED, kw
    assert glu(lib, M=0, x=None, h=None, a=None, q=None, qt=None) == ERR_UNSUPPORTED


@pytest.mark.parametrize("act", [3, 4])
def test_the_plain_calls_refuse_the_gated_activations(lib, act):
    assert lib.fp8_quant_fused(A, 64, 256, act, 0, A, A, A, None, A, A, None, 1, None) == ERR_UNSUPPORTED
    assert lib.fp8_upproj_fwd(A, A, A, A, act, A, A, A, A, A, A, 64, 64, 64, 0, None, None) == ERR_UNSUPPORTED
    assert lib.fp8_gemm_dgrad_act(A, A, A, A, A, act, A, 64, 64, 64, None, None) == ERR_UNSUPPORTED


def struct_call(fn, cls, base):
    def call(**kw):
        a = cls()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return fn(ctypes.byref(a), None)
    return call


@pytest.fixture
def fwd(lib):
    return struct_call(lib.block_norm_fwd, B.BlockNormArgs, dict(
        M=8, N=64, dtype=B.BF16, param_dtype=B.FP32, x=A, ldx=64, residual=A, ld_residual=64, r_out=A, ld_r=64, y=A, ldy=64, weight=A,
        post_weight=A, gate=A, alpha=A, rstd=A, rstd_post=A, eps=1e-5, post_norm=1))


@pytest.fixture
def bwd(lib):
    return struct_call(lib.block_norm_bwd, B.BlockNormBwdArgs, dict(
        M=8, N=64, dtype=B.FP16, param_dtype=B.FP16, dy=A, ld_dy=64, r=A, ld_r=64, dr=A, ld_dr=64, x=A, ldx=64, residual=A, ld_residual=64,
        dresidual=A, ld_dresidual=64, dx=A, ld_dx=64, weight=A, post_weight=A, gate=A, alpha=A, rstd=A, rstd_post=A, dweight=A,
        dpost_weight=A, dgate=A, dalpha=A, workspace=A, workspace_bytes=1 << 20, post_norm=1))


def test_block_norm_fwd_argument_checks(lib, fwd):
    assert lib.block_norm_fwd(None, None) == ERR_NULL
    assert fwd(x=None) == ERR_NULL and fwd(y=None, r_out=None) == ERR_NULL
    assert fwd(q_out=A) == ERR_NULL and fwd(amax_out=A) == ERR_NULL  # no scale
    for bad in (3, -1):
        assert fwd(dtype=bad) == ERR_UNSUPPORTED
    assert fwd(param_dtype=B.FP16) == ERR_UNSUPPORTED and fwd(flags=2) == ERR_UNSUPPORTED
    assert fwd(q_out=A, scale=A, fmt=2) == ERR_UNSUPPORTED
    for k in ("M", "N", "ldx", "ldy", "ld_r", "ld_residual"):
        assert fwd(**{k: -1}) == ERR_SHAPE, k
    assert fwd(N=0) == ERR_SHAPE and fwd(M=1 << 31) == ERR_SHAPE and fwd(ld_residual=63) == ERR_SHAPE
    for eps in (-1e-5, float("inf"), float("nan")):
        assert fwd(eps=eps) == ERR_SHAPE
    for k in ("x", "residual", "r_out", "y", "weight", "post_weight", "gate", "alpha", "rstd", "rstd_post"):
        assert fwd(**{k: A + 1}) == ERR_ALIGN, k
    assert fwd(q_out=A, scale=A, sat_count=A + 4) == ERR_ALIGN


def test_block_norm_bwd_argument_checks(lib, bwd):
    assert lib.block_norm_bwd(None, None) == ERR_NULL
    for k in ("r", "rstd", "x", "rstd_post", "residual", "workspace"):
        assert bwd(**{k: None}) == ERR_NULL, k
    assert bwd(dy=None) == ERR_NULL  # dweight without a norm
    assert bwd(dy=None, dr=None, dweight=None) == ERR_NULL
    assert bwd(dresidual=None, dx=None, dweight=None, dpost_weight=None, dgate=None, dalpha=None) == ERR_NULL
    assert bwd(dtype=7) == ERR_UNSUPPORTED and bwd(param_dtype=B.BF16) == ERR_UNSUPPORTED and bwd(flags=4) == ERR_UNSUPPORTED
    assert bwd(N=0) == ERR_SHAPE and bwd(M=-1) == ERR_SHAPE and bwd(N=1 << 31) == ERR_SHAPE
    for k in ("ld_dy", "ld_r", "ld_dr", "ldx", "ld_residual", "ld_dresidual", "ld_dx"):
        assert bwd(**{k: 63}) == ERR_SHAPE, k
    for k in ("dy", "r", "dr", "x", "residual", "dresidual", "dx", "weight", "post_weight", "gate", "alpha", "rstd", "rstd_post", "dweight",
              "dpost_weight", "dgate", "dalpha", "workspace"):
        assert bwd(**{k: A + 1}) == ERR_ALIGN, k


@no_gpu
def test_block_norm_well_formed(lib, fwd, bwd):
    for kw in ({}, dict(y=None, rstd=None), dict(y=None, r_out=None, q_out=A, scale=A), dict(residual=None, alpha=None), dict(M=0, x=None),
               dict(eps=0.0), dict(weight=None, post_weight=None, gate=None), dict(x=A + 2)):
        assert fwd(**kw) == ERR_UNSUPPORTED, kw
    for kw in ({}, dict(dy=None, r=None, rstd=None, weight=None, dweight=None), dict(dr=None), dict(dalpha=None, residual=None),
               dict(x=None, dx=None, dpost_weight=None, dgate=None), dict(post_norm=0, rstd_post=None),
               dict(M=0, dy=None, dr=None, workspace=None)):
        assert bwd(**kw) == ERR_UNSUPPORTED, kw


def test_block_norm_workspace_bytes(lib):
    f = lib.block_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(1 << 31, 4) == 0 and f(4, 1 << 31) == 0
    for M in (1, 2, 63, 64, 1000, 131072, 2 ** 31 - 1):
        for N in (1, 64, 768, 1601, 16384, 100000):
            assert 4 * (2 * N + 1) <= f(M, N) <= 1024 * (8 * N + 4) and f(M, N) % 16 == 0


def test_binding_refuses_host_tensors_and_shapes():
    x, w, f = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16), torch.ones(1)
    q, w1 = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(32, 16, dtype=torch.uint8)
    with pytest.raises(TypeError):
        B.block_norm_fwd(x, w, x)
    with pytest.raises(TypeError):
        B.block_norm_fwd(x.double(), w, x)
    with pytest.raises(TypeError):
        B.block_norm_bwd(x, x, torch.ones(4), w, dresidual=x)
    with pytest.raises(TypeError):
        B.block_norm_bwd(None, None, None, None, dresidual=x)
    with pytest.raises(TypeError):
        B.fp8_glu_fwd(q, w1, f, f, act_out=x)
    with pytest.raises(TypeError):
        B.fp8_glu_fwd(q[0], w1, f, f, act_out=x)
    with pytest.raises(ValueError, match="rows"):
        B.fp8_glu_fwd(q, w1[:31], f, f, act_out=x)
    with pytest.raises(TypeError):
        B.fp8_gemm_dgrad_glu(q, w1, f, f, x, dh=x)


@pytest.mark.parametrize("form,cls", [(B._block_norm, B.BlockNormArgs), (B._block_norm_bwd, B.BlockNormBwdArgs),
                                      (B._glu, B.GluArgs), (B._glu, B.DgradGluArgs)])
def test_packed_arguments_are_the_structs(form, cls):
    """The bytes that the binding packs, field by field the ctypes structure's."""
    values = [0.5 if t is ctypes.c_float else 1000 + i if t is not ctypes.c_int else i % 3 for i, (_, t) in enumerate(cls._fields_)]
    got = cls.from_buffer_copy(form.pack(*values))
    assert [getattr(got, n) for n, _ in cls._fields_] == values


@pytest.fixture(scope="module")
def stack():
    from quantize_fp8_gemm_gb300 import build
    build.build()
    return Fp8GatedMlpStack(32, 16, 48, 2, device="cpu")


def layer(**kw):
    p = dict(weight=torch.ones(16), post=torch.ones(16), alpha=None, w1=torch.zeros(16, 96, dtype=torch.bfloat16),
             w2=torch.zeros(48, 16, dtype=torch.bfloat16))
    return tuple({**p, **kw}.values())


def test_stack_checks_its_parameters(stack):
    x = torch.zeros(32, 16, dtype=torch.bfloat16)
    for call in (stack.forward, stack.backward):
        for count in (0, 1, 3):
            with pytest.raises(ValueError, match="2 sub-layers"):
                call(x, [layer() for _ in range(count)])
        with pytest.raises(ValueError, match="1 gates for 2 sub-layers"):
            call(x, [layer(), layer()], [None])
        with pytest.raises(ValueError, match="W1"):
            call(x, [layer(), layer(w1=torch.zeros(96, 16, dtype=torch.bfloat16))])
        with pytest.raises(TypeError, match="W2 must be torch.bfloat16"):
            call(x, [layer(w2=torch.zeros(48, 16)), layer()])
    for bad in (dict(M=100), dict(D=100), dict(K=100), dict(layers=0)):
        with pytest.raises(ValueError):
            Fp8GatedMlpStack(**{**dict(M=64, D=64, K=64, layers=1), **bad})
