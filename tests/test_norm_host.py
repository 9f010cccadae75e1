"""Layer norm and dropout without a GPU: the tests' own 64-bit reference against known
answers, and the argument checks of the C entry points and of the binding.  No kernel
is launched; the pointers passed here are never dereferenced."""
import ctypes

import numpy as np
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from tests import norm_reference as R

OK, ERR_NULL, ERR_ALIGN, ERR_SHAPE, ERR_UNSUPPORTED, ERR_CUDA = range(6)
A = 1 << 20  # an aligned fake device address
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a well-formed call would launch on the fake addresses")


@pytest.fixture(scope="module")
def lib():
    from quantize_fp8_gemm_gb300 import build
    build.build()
    return B.lib()


def test_philox_known_answers():
    """The published known-answer vectors of Philox4x32-10 (counter, key -> words)."""
    for ctr, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        assert tuple(int(v) for v in R.philox(ctr, key)) == want


def test_mask_rate_and_independence():
    a = R.keep_mask(7, 1, 400, 1000, 0.3)
    assert abs(a.mean() - 0.7) < 5 * np.sqrt(0.21 / a.size)
    b = R.keep_mask(7, 2, 400, 1000, 0.3)
    assert abs((a & b).mean() - 0.49) < 5 * np.sqrt(0.25 / a.size)
    assert np.array_equal(a[100:], R.keep_mask(7, 1, 300, 1000, 0.3, row0=100))


def test_reference_against_autograd():
    rng = np.random.default_rng(3)
    r, dy, w, b = (torch.from_numpy(rng.standard_normal(s)) for s in ((5, 33), (5, 33), 33, 33))
    r.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    y = torch.nn.functional.layer_norm(r, (33,), w, b, 1e-5)
    y.backward(dy)
    y64, mean, rstd = R.norm_fwd(R.f64(r), R.f64(w), R.f64(b), 1e-5)
    assert np.allclose(y64, R.f64(y), rtol=1e-12, atol=1e-13)
    dr, dw, db = R.norm_bwd(R.f64(dy), R.f64(r), mean, rstd, R.f64(w), None)
    for got, want in ((dr, r.grad), (dw, w.grad), (db, b.grad)):
        assert np.allclose(got, R.f64(want), rtol=1e-10, atol=1e-11)


def fwd(lib, **kw):
    a = B.LayerNormArgs()
    base = dict(M=8, N=64, dtype=B.BF16, param_dtype=B.FP32, x=A, ldx=64, weight=A, bias=A, y=A, ldy=64, mean=A, rstd=A,
                eps=1e-5)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return lib.layer_norm_fwd(ctypes.byref(a), None)


def test_layer_norm_fwd_argument_checks(lib):
    assert lib.layer_norm_fwd(None, None) == ERR_NULL
    assert fwd(lib, x=None) == ERR_NULL
    assert fwd(lib, y=None) == ERR_NULL
    assert fwd(lib, q_out=A) == ERR_NULL  # no scale
    assert fwd(lib, amax_out=A) == ERR_NULL
    assert fwd(lib, p=0.1) == ERR_NULL  # no rng
    for bad in (3, -1):
        assert fwd(lib, dtype=bad) == ERR_UNSUPPORTED
    assert fwd(lib, param_dtype=B.FP16) == ERR_UNSUPPORTED
    assert fwd(lib, flags=2) == ERR_UNSUPPORTED
    assert fwd(lib, q_out=A, scale=A, fmt=2) == ERR_UNSUPPORTED
    for k in ("M", "N", "ldx", "ldy"):
        assert fwd(lib, **{k: -1}) == ERR_SHAPE
    assert fwd(lib, N=0) == ERR_SHAPE
    assert fwd(lib, M=1 << 31) == ERR_SHAPE
    assert fwd(lib, ldx=63) == ERR_SHAPE and fwd(lib, ldy=63) == ERR_SHAPE
    assert fwd(lib, residual=A, ld_residual=63) == ERR_SHAPE
    assert fwd(lib, r_out=A, ld_r=0) == ERR_SHAPE
    for p in (-0.1, 1.1, float("nan")):
        assert fwd(lib, p=p, rng=A) == ERR_SHAPE
    for eps in (-1e-5, float("inf"), float("nan")):
        assert fwd(lib, eps=eps) == ERR_SHAPE
    for k in ("x", "y", "weight", "mean", "rstd"):
        assert fwd(lib, **{k: A + 1}) == ERR_ALIGN
    assert fwd(lib, weight=A + 2) == ERR_ALIGN  # float32 parameters
    assert fwd(lib, p=0.1, rng=A + 4) == ERR_ALIGN
    assert fwd(lib, q_out=A, scale=A, sat_count=A + 4) == ERR_ALIGN


@no_gpu
def test_layer_norm_fwd_well_formed(lib):
    """Only the device check remains, and there is no sm_103 here."""
    for kw in ({}, dict(x=A + 2), dict(y=None, q_out=A, scale=A), dict(weight=None, bias=None), dict(p=1.0, rng=A),
               dict(p=1e-11), dict(M=0, x=None, y=None), dict(eps=0.0), dict(N=1), dict(param_dtype=B.BF16, weight=A + 2)):
        assert fwd(lib, **kw) == ERR_UNSUPPORTED, kw


def bwd(lib, **kw):
    a = B.LayerNormBwdArgs()
    base = dict(M=8, N=64, dtype=B.FP16, param_dtype=B.FP16, dy=A, ld_dy=64, r=A, ld_r=64, mean=A, rstd=A, weight=A,
                dx=A, ld_dx=64, dweight=A, dbias=A, workspace=A, workspace_bytes=1 << 20)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return lib.layer_norm_bwd(ctypes.byref(a), None)


def test_layer_norm_bwd_argument_checks(lib):
    assert lib.layer_norm_bwd(None, None) == ERR_NULL
    for k in ("dy", "r", "mean", "rstd", "dx", "workspace"):
        assert bwd(lib, **{k: None}) == ERR_NULL, k
    assert bwd(lib, dbranch=A, ld_dbranch=64, p=0.5) == ERR_NULL
    assert bwd(lib, dtype=7) == ERR_UNSUPPORTED
    assert bwd(lib, param_dtype=B.BF16) == ERR_UNSUPPORTED
    assert bwd(lib, flags=4) == ERR_UNSUPPORTED
    assert bwd(lib, N=0) == ERR_SHAPE and bwd(lib, M=-1) == ERR_SHAPE and bwd(lib, N=1 << 31) == ERR_SHAPE
    for k in ("ld_dy", "ld_r", "ld_dx"):
        assert bwd(lib, **{k: 63}) == ERR_SHAPE
    assert bwd(lib, dresidual=A, ld_dresidual=63) == ERR_SHAPE
    assert bwd(lib, dbranch=A, ld_dbranch=63) == ERR_SHAPE
    assert bwd(lib, p=2.0, rng=A) == ERR_SHAPE
    assert bwd(lib, workspace_bytes=lib.layer_norm_bwd_workspace_bytes(8, 64) - 1) == ERR_SHAPE
    for k in ("dy", "r", "dx", "weight", "mean", "rstd", "dweight", "dbias", "workspace"):
        assert bwd(lib, **{k: A + 1}) == ERR_ALIGN, k
    assert bwd(lib, workspace=A + 8) == ERR_ALIGN


@no_gpu
def test_layer_norm_bwd_well_formed(lib):
    for kw in ({}, dict(weight=None), dict(dweight=None, dbias=None, workspace=None, workspace_bytes=0),
               dict(dbranch=A, ld_dbranch=64), dict(M=0, dy=None, r=None, mean=None, rstd=None, dx=None, workspace=None)):
        assert bwd(lib, **kw) == ERR_UNSUPPORTED, kw


def test_workspace_bytes(lib):
    f = lib.layer_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(1 << 31, 4) == 0 and f(4, 1 << 31) == 0
    for M in (1, 2, 63, 64, 1000, 131072, 2 ** 31 - 1):
        for N in (1, 64, 768, 1601, 16384, 100000):
            assert 0 < f(M, N) <= 8192 * N and f(M, N) % (8 * N) == 0


def drop(lib, x=A, ldx=64, res=None, ldr=0, y=A, ldy=64, M=8, N=64, dtype=0, p=0.1, rng=A):
    return lib.dropout_fwd(x, ldx, res, ldr, y, ldy, M, N, dtype, p, rng, None)


def test_dropout_argument_checks(lib):
    assert drop(lib, x=None) == ERR_NULL and drop(lib, y=None) == ERR_NULL and drop(lib, rng=None) == ERR_NULL
    assert drop(lib, dtype=3) == ERR_UNSUPPORTED
    assert drop(lib, M=-1) == ERR_SHAPE and drop(lib, N=0) == ERR_SHAPE and drop(lib, M=1 << 31) == ERR_SHAPE
    assert drop(lib, ldx=63) == ERR_SHAPE and drop(lib, ldy=63) == ERR_SHAPE and drop(lib, res=A, ldr=63) == ERR_SHAPE
    assert drop(lib, p=-1.0) == ERR_SHAPE and drop(lib, p=float("nan")) == ERR_SHAPE
    assert drop(lib, x=A + 1) == ERR_ALIGN and drop(lib, y=A + 1) == ERR_ALIGN and drop(lib, rng=A + 4) == ERR_ALIGN
    assert drop(lib, dtype=2, x=A + 2) == ERR_ALIGN
    assert lib.dropout_bwd(None, 64, A, 64, 8, 64, 0, 0.1, A, None) == ERR_NULL
    assert lib.dropout_bwd(A, 63, A, 64, 8, 64, 0, 0.1, A, None) == ERR_SHAPE
    assert lib.dropout_bwd(A, 64, A, 64, 8, 64, 0, 1.5, A, None) == ERR_SHAPE


@no_gpu
def test_dropout_well_formed(lib):
    assert drop(lib) == ERR_UNSUPPORTED and drop(lib, p=0.0, rng=None) == ERR_UNSUPPORTED
    assert drop(lib, M=0, x=None, y=None) == ERR_UNSUPPORTED
    assert lib.dropout_bwd(A, 64, A, 64, 8, 64, 0, 0.1, A, None) == ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(TypeError):
        B.layer_norm_fwd(x, w, w, x)
    with pytest.raises(TypeError):
        B.layer_norm_fwd(x[0], w, w, x)
    with pytest.raises(TypeError):
        B.layer_norm_fwd(x.double(), w, w, x)
    with pytest.raises(TypeError):
        B.layer_norm_bwd(x, x, w, w, w, x)
    with pytest.raises(TypeError):
        B.dropout_fwd(x, x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        B.dropout_bwd(x, x, 0.1, torch.zeros(2, dtype=torch.int64))
