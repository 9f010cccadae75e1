"""layer_norm_fwd / layer_norm_bwd and dropout_fwd / dropout_bwd on the GPU against the
64-bit reference of tests/norm_reference.py, with the tolerances derived there.  What is
discrete is exact: dropout masks, the stored residual stream r, FP8 codes, amax,
saturation counts, and the fused calls against the separate ones."""
import numpy as np
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from tests import norm_reference as R
from tests.norm_reference import assert_within, f64

pytestmark = pytest.mark.gpu

BF, HF, SF = torch.bfloat16, torch.float16, torch.float32
ids = {BF: "bf16", HF: "fp16", SF: "fp32"}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(M, N, T, seed, std=1.0, mean=0.0, pad=0, shift=0):
    """[M, N] on the GPU whose rows are N + pad apart and start `shift` elements into the buffer."""
    host = (torch.randn(M, N, generator=gen(seed)) * std + mean).to(T)
    buf = torch.full((M * (N + pad) + shift + 16,), float("nan"), dtype=T, device="cuda")
    view = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(host)
    return view


def out_like(M, N, T, pad=0, shift=0):
    return rows(M, N, T, 0, std=0.0, mean=7.0, pad=pad, shift=shift)


def padding_untouched(t):
    """The elements between the rows of a rows() view are still NaN."""
    M, N = t.shape
    ld = t.stride(0)
    if ld == N or M < 2:
        return True
    gaps = torch.as_strided(t, (M - 1, ld - N), (ld, 1), t.storage_offset() + N)
    return bool(gaps.isnan().all())


def rng_of(seed, offset):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


def params(N, T, seed):
    w = (1.0 + 0.3 * torch.randn(N, generator=gen(seed))).to(T).cuda()
    b = (0.2 * torch.randn(N, generator=gen(seed + 1))).to(T).cuda()
    return w, b


def check_fwd(x, w, b, eps=1e-5, y=None, **kw):
    M, N = x.shape
    T = x.dtype
    y = out_like(M, N, T) if y is None else y
    mean, rstd = torch.full((M,), 9.0, device="cuda"), torch.full((M,), 9.0, device="cuda")
    r = f64(x)
    B.layer_norm_fwd(x, w, b, y, eps=eps, mean=mean, rstd=rstd, **kw)
    torch.cuda.synchronize()
    w64, b64 = (f64(w) if w is not None else np.ones(N)), (f64(b) if b is not None else np.zeros(N))
    want = R.norm_fwd(r, w64, b64, eps)
    tol = R.fwd_tolerances(r, w64, b64, eps, T)
    for got, v, t, name in zip((y, mean, rstd), want, tol, ("y", "mean", "rstd")):
        assert_within(f64(got), v, t, name)
    assert padding_untouched(y)
    return y, mean, rstd


SIZES = [(1, 1), (3, 2), (2, 3), (5, 4), (7, 7), (4, 8), (33, 16), (9, 31), (64, 64), (5, 100), (17, 127), (3, 128),
         (130, 129), (10, 255), (6, 256), (40, 768), (11, 1001), (9, 1024), (37, 1600), (5, 2047), (4, 2048), (3, 2056),
         (4, 4096), (3, 4099), (5, 6400), (2, 8191), (3, 8192), (2, 12345), (3, 16384), (2, 16392), (2, 32768), (2, 40000),
         (2, 65536)]


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N", SIZES)
def test_fwd_sizes(M, N, T):
    w, b = params(N, SF if (M + N) % 2 else T, N)
    check_fwd(rows(M, N, T, M * N, std=2.0, mean=0.5), w, b)


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N,pad,shift", [(5, 64, 8, 0), (5, 64, 3, 0), (6, 768, 16, 8), (6, 768, 0, 1), (4, 1600, 1, 0),
                                           (3, 1001, 6, 5), (3, 4096, 2, 2), (4, 3, 1, 1), (2, 20000, 5, 3)])
def test_fwd_layouts(M, N, pad, shift, T):
    """Row strides and base addresses that are and are not multiples of 16 bytes, in x and in y alone."""
    w, b = params(N, T, 5)
    x = rows(M, N, T, 77, pad=pad, shift=shift)
    check_fwd(x, w, b, y=out_like(M, N, T, pad=pad, shift=shift))
    check_fwd(x, w, b)
    check_fwd(rows(M, N, T, 78), w, b, y=out_like(M, N, T, pad=pad, shift=shift))
    wide, _ = params(N + 1, T, 6)
    check_fwd(rows(M, N, T, 79), wide[1:], None)  # a parameter vector off the 16-byte grid


@pytest.mark.parametrize("T", [BF, SF], ids=ids.get)
@pytest.mark.parametrize("N", [64, 1001, 1600, 2056, 40000])
def test_fwd_no_params_and_optional_outputs(N, T):
    x = rows(5, N, T, 1)
    y, mean, rstd = check_fwd(x, None, None)
    y2 = out_like(5, N, T)
    B.layer_norm_fwd(x, None, None, y2)
    assert torch.equal(y, y2)
    _, b = params(N, T, 2)
    check_fwd(x, None, b)


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("N", [1, 64, 1001, 1600, 2056, 40000])
def test_fwd_hard_rows(N, T):
    """Rows of one value, zeros, a far mean, the type's largest and smallest values; and NaN or
    infinity, which stay in their own rows."""
    x = rows(12, N, T, 3)
    big = {BF: 1e18, HF: 60000.0, SF: 1e18}[T]
    x[1] = 0.0
    x[2] = 0.1
    x[3] += 1000.0
    x[4] = big
    x[5] = -big
    x[6, :] = 0.0
    x[6, N // 2] = big
    x[7] *= 1e-7 if T == HF else 1e-30
    w, b = params(N, SF, 4)
    check_fwd(x, w, b)
    y, mean, rstd = out_like(12, N, T), torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
    B.layer_norm_fwd(x, w, b, y)
    x[8, N // 3] = float("nan")
    x[9, 0] = float("inf")
    x[10, N - 1] = float("-inf")
    y2 = out_like(12, N, T)
    B.layer_norm_fwd(x, w, b, y2, mean=mean, rstd=rstd)
    assert y2[8:11].isnan().all() and mean[8].isnan() and mean[9].isinf() and mean[10].isinf()
    keep = [i for i in range(12) if i not in (8, 9, 10)]
    assert torch.equal(y2[keep], y[keep])


@pytest.mark.parametrize("N", [16, 768, 1001, 2056, 33000])
@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-3, 10.0])
def test_fwd_eps(N, eps):
    w, b = params(N, SF, 8)
    check_fwd(rows(7, N, SF, 9, std=0.01), w, b, eps=eps)


@pytest.mark.parametrize("fmt", [B.E4M3, B.E5M2])
@pytest.mark.parametrize("M,N", [(1, 16), (64, 64), (33, 768), (9, 1600), (5, 1001), (3, 4096), (2, 40000), (3, 7)])
def test_fwd_codes_bit_exact(M, N, fmt):
    """q, amax and the saturation count are the framework's own cast of the y that the call returns."""
    x = rows(M, N, BF, 21, pad=3 if N % 2 else 0)
    w, b = params(N, SF, 22)
    y = out_like(M, N, BF)
    q = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")
    amax, sat = torch.full((1,), 99.0, device="cuda"), torch.full((1,), 99, dtype=torch.int64, device="cuda")
    scale = torch.full((1,), 300.0 if fmt == B.E4M3 else 40000.0, device="cuda")
    B.layer_norm_fwd(x, w, b, y, fmt=fmt, scale=scale, q_out=q, amax_out=amax, sat_count=sat)
    q2 = B.fp8_cast_f32((y.float() * scale).contiguous(), fmt)
    assert torch.equal(q, q2)
    assert amax.item() == y.float().abs().max().item()
    want = int((y.float() * scale).abs().gt(448.0 if fmt == B.E4M3 else 57344.0).sum())
    assert sat.item() == want and (want > 0 or M * N < 100)
    if N % 16 == 0:
        q3, a3, s3 = torch.empty_like(q), torch.zeros_like(amax), torch.zeros_like(sat)
        B.fp8_quant_fused(y, B.ACT_IDENTITY, fmt, scale, q_out=q3, amax_out=a3, sat_count=s3)
        assert torch.equal(q, q3) and a3.item() == amax.item() and s3.item() == sat.item()
    # codes alone (y not kept), and accumulating counters
    q4 = torch.empty_like(q)
    B.layer_norm_fwd(x, w, b, None, fmt=fmt, scale=scale, q_out=q4, amax_out=amax, sat_count=sat, flags=B.ACCUMULATE)
    assert torch.equal(q, q4) and sat.item() == 2 * want and amax.item() == y.float().abs().max().item()
    amax.fill_(1e9)
    B.layer_norm_fwd(x, w, b, y, fmt=fmt, scale=scale, amax_out=amax, flags=B.ACCUMULATE)
    assert amax.item() == 1e9


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("N", [5, 64, 200, 1000, 1600, 2048, 3000, 6400, 16384, 20000])
def test_results_do_not_depend_on_where_rows_lie(N, T):
    """Rows on and off the 16-byte grid give the same bits (the column sums may differ in order)."""
    M = 21
    w, b = params(N, SF, 1)
    rng = rng_of(3, 4)
    seen = []
    for pad, shift in ((0, 0), (3, 0), (1, 5), (8, 16)):
        x, res, dy, dres = (rows(M, N, T, s, pad=pad, shift=shift) for s in (1, 2, 3, 4))
        r, y, dx, db = (out_like(M, N, T, pad=pad, shift=shift) for _ in range(4))
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        B.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, residual=res, r_out=r, p=0.2, rng=rng)
        run_bwd(dy, r, mean, rstd, w, dres=dres, p=0.2, rng=rng, dx=dx, db=db)
        seen.append([t.clone() for t in (r, y, mean, rstd, dx, db)])
    for other in seen[1:]:
        assert all(torch.equal(a, c) for a, c in zip(seen[0], other))


def test_fwd_amax_of_a_nan():
    x = rows(4, 64, BF, 1)
    x[2, 5] = float("nan")
    q, amax = torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    B.layer_norm_fwd(x, None, None, None, scale=torch.ones(1, device="cuda"), q_out=q, amax_out=amax)
    assert amax.isnan().all()


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N,pad", [(1, 1, 0), (3, 5, 0), (64, 64, 0), (37, 1025, 0), (9, 1600, 8), (5, 1001, 6),
                                     (4, 2056, 1), (3, 33000, 0), (70, 333, 3)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout_exact(M, N, pad, p, T):
    x, res = rows(M, N, T, 31, pad=pad), rows(M, N, T, 32, std=2.0, pad=pad)
    seed, off = 0xDEADBEEF12345678, 0xFEDCBA9876543210
    rng = rng_of(seed, off)
    keep = R.keep_mask(seed, off, M, N, p)
    for residual in (None, res):
        y = out_like(M, N, T, pad=pad)
        B.dropout_fwd(x, y, p, rng, residual=residual)
        want = R.residual_stream(x.cpu(), None if residual is None else residual.cpu(), keep, p)
        assert torch.equal(y.cpu(), want) and padding_untouched(y)
    dx = out_like(M, N, T, pad=pad)
    B.dropout_bwd(x, dx, p, rng)
    assert torch.equal(dx.cpu(), R.residual_stream(x.cpu(), None, keep, p)) and padding_untouched(dx)


def test_dropout_drops_what_is_not_finite():
    x = torch.full((8, 64), float("inf"), dtype=BF, device="cuda")
    x[4:] = float("nan")
    y = torch.empty_like(x)
    keep = torch.from_numpy(R.keep_mask(5, 6, 8, 64, 0.5)).cuda()
    B.dropout_fwd(x, y, 0.5, rng_of(5, 6))
    assert (y[~keep] == 0).all() and not y[keep].isfinite().any()
    B.dropout_fwd(x, y, 1.0, rng_of(5, 6), residual=torch.ones_like(x))
    assert (y == 1).all()
    # a p below half a word drops nothing and needs no generator
    x = rows(8, 64, BF, 1)
    B.dropout_fwd(x, y, 1e-11, None)
    assert torch.equal(x, y)


def test_mask_depends_on_position_alone():
    """The same mask for every type, layout and kernel, and for a block of the columns' left part."""
    rng, p = rng_of(11, 12), 0.4
    masks = []
    for T in (BF, HF, SF):
        for pad, shift in ((0, 0), (3, 1), (16, 8)):
            x = rows(20, 1600, T, 1, pad=pad, shift=shift)
            x.fill_(1.0)
            y = out_like(20, 1600, T, pad=pad, shift=shift)
            B.dropout_fwd(x, y, p, rng)
            masks.append(y != 0)
            r = out_like(20, 1600, T, pad=pad, shift=shift)
            B.layer_norm_fwd(x, None, None, y, r_out=r, p=p, rng=rng)
            masks.append(r != 0)
    x = torch.ones(20, 1003, dtype=BF, device="cuda")
    y = torch.empty_like(x)
    B.dropout_fwd(x, y, p, rng)
    assert all(torch.equal(m, masks[0]) for m in masks)
    assert torch.equal(y != 0, masks[0][:, :1003])


FUSED = [(1, 1, 0), (3, 7, 0), (64, 64, 0), (33, 768, 0), (9, 1600, 8), (5, 1001, 6), (4, 2056, 0), (3, 4099, 0),
         (3, 6400, 1), (2, 16384, 0), (2, 33000, 0), (150, 1024, 0)]


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N,pad", FUSED)
def test_fused_forward_equals_the_separate_calls(M, N, pad, T):
    x, res = rows(M, N, T, 41, pad=pad), rows(M, N, T, 42, std=2.0, pad=pad)
    w, b = params(N, T, 43)
    seed, off = 1 << 63 | 17, 3
    rng = rng_of(seed, off)
    for p, residual in ((0.1, res), (0.3, None), (0.0, res), (1.0, res)):
        keep = R.keep_mask(seed, off, M, N, p) if p else None
        r_want = R.residual_stream(x.cpu(), None if residual is None else residual.cpu(), keep, p)
        r, y = out_like(M, N, T, pad=pad), out_like(M, N, T, pad=pad)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        B.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, residual=residual, r_out=r, p=p, rng=rng)
        assert torch.equal(r.cpu(), r_want) and padding_untouched(r)
        y2, mean2, rstd2 = check_fwd(r, w, b, y=out_like(M, N, T, pad=pad))
        assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
        y3 = out_like(M, N, T)  # r not kept
        B.layer_norm_fwd(x, w, b, y3, residual=residual, p=p, rng=rng)
        assert_within(f64(y3), f64(y), 2 * R.fwd_tolerances(f64(r), f64(w), f64(b), 1e-5, T)[0], "y without r_out")


@pytest.mark.parametrize("N", [64, 1600, 1001, 2056, 16384, 33000])
@pytest.mark.parametrize("p", [0.0, 1e-11])
def test_r_out_of_a_call_without_residual_or_dropout(N, p):
    """r is x then, and r_out gets it; so also where p is too small to drop anything."""
    x = rows(6, N, BF, 55)
    r, y, y2 = (out_like(6, N, BF) for _ in range(3))
    B.layer_norm_fwd(x, None, None, y, r_out=r, p=p)
    B.layer_norm_fwd(x, None, None, y2)
    assert torch.equal(r, x) and torch.equal(y, y2)


@pytest.mark.parametrize("N", [64, 1600, 1001, 2056, 33000])
def test_forward_in_place(N):
    """r_out over the residual, y over the branch: as a program without spare buffers calls it."""
    x, res = rows(6, N, BF, 51), rows(6, N, BF, 52)
    w, b = params(N, SF, 53)
    rng = rng_of(9, 9)
    r, y = out_like(6, N, BF), out_like(6, N, BF)
    B.layer_norm_fwd(x, w, b, y, residual=res, r_out=r, p=0.2, rng=rng)
    B.layer_norm_fwd(x, w, b, x, residual=res, r_out=res, p=0.2, rng=rng)
    assert torch.equal(x, y) and torch.equal(res, r)
    d, want = rows(6, N, BF, 54), out_like(6, N, BF)
    B.dropout_fwd(d, want, 0.2, rng, residual=r)
    B.dropout_fwd(d, d, 0.2, rng, residual=r)
    assert torch.equal(d, want)


def run_bwd(dy, r, mean, rstd, w, *, dres=None, p=0.0, rng=None, want_branch=False, dx=None, db=None, flags=0,
            dweight=None, dbias=None):
    M, N = dy.shape
    dx = out_like(M, N, dy.dtype) if dx is None else dx
    if db is None and want_branch:
        db = out_like(M, N, dy.dtype)
    dweight = torch.full((N,), 3.0, device="cuda") if dweight is None else dweight
    dbias = torch.full((N,), 3.0, device="cuda") if dbias is None else dbias
    n = B.layer_norm_bwd_workspace_bytes(M, N)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs: nothing may be read unwritten
    B.layer_norm_bwd(dy, r, mean, rstd, w, dx, dresidual=dres, dweight=dweight, dbias=dbias, workspace=ws[:n], p=p,
                     rng=rng, dbranch=db, flags=flags)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xFF).all()
    return dx, db, dweight, dbias


def stats(r, eps=1e-5):
    r = r.double()
    mean = r.mean(1)
    return mean.float(), (1.0 / ((r - mean[:, None]).square().mean(1) + eps).sqrt()).float()


def check_bwd(dy, r, w, dres=None, p=0.0, seed=1, off=2, want_branch=False, **kw):
    M, N = dy.shape
    T = dy.dtype
    mean, rstd = stats(r)
    dx, db, dweight, dbias = run_bwd(dy, r, mean, rstd, w, dres=dres, p=p, rng=rng_of(seed, off) if p else None,
                                     want_branch=want_branch, **kw)
    w64 = f64(w) if w is not None else np.ones(N)
    args = (f64(dy), f64(r), f64(mean), f64(rstd), w64, None if dres is None else f64(dres))
    dr, dw, dbs = R.norm_bwd(*args)
    inv = 1.0 / (1.0 - p) if p < 1 else 0.0
    t_dx, t_db, t_dw, t_dbias = R.bwd_tolerances(*args, T, inv)
    assert_within(f64(dx), dr, t_dx, "dx")
    assert_within(f64(dweight), dw, t_dw, "dweight")
    assert_within(f64(dbias), dbs, t_dbias, "dbias")
    assert padding_untouched(dx)
    if want_branch:
        keep = R.keep_mask(seed, off, M, N, p) if p else np.ones((M, N), bool)
        assert (f64(db)[~keep] == 0).all()
        assert_within(f64(db), np.where(keep, dr * inv, 0.0), t_db, "dbranch")
        assert padding_untouched(db)
    return dx, db, dweight, dbias


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N", SIZES + [(1000, 64), (700, 768), (333, 1001), (300, 1600), (2500, 8), (3000, 3)])
def test_bwd_sizes(M, N, T):
    w, _ = params(N, SF if (M + N) % 2 else T, N)
    dy, r = rows(M, N, T, 61), rows(M, N, T, 62, std=2.0, mean=0.3)
    check_bwd(dy, r, w)
    check_bwd(dy, r, w, dres=rows(M, N, T, 63), p=0.1, want_branch=True)


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N,pad,shift", [(50, 64, 8, 0), (50, 64, 3, 0), (60, 768, 16, 8), (60, 768, 0, 1), (40, 1600, 1, 0),
                                           (30, 1001, 6, 5), (30, 4096, 2, 2), (40, 3, 1, 1), (20, 20000, 5, 3),
                                           (6, 33000, 8, 0)])
def test_bwd_layouts(M, N, pad, shift, T):
    w, _ = params(N, T, 5)
    dy, r, dres = (rows(M, N, T, s, pad=pad, shift=shift) for s in (71, 72, 73))
    out = lambda: out_like(M, N, T, pad=pad, shift=shift)  # noqa: E731
    check_bwd(dy, r, w, dres=dres, p=0.25, want_branch=True, dx=out(), db=out())
    check_bwd(dy, r, w, dres=dres, want_branch=True)  # p = 0: dbranch is dr rounded
    wide, _ = params(N + 1, T, 6)
    check_bwd(rows(M, N, T, 74), rows(M, N, T, 75), wide[1:], dx=out())


@pytest.mark.parametrize("N", [64, 1001, 1600, 2056, 33000])
def test_bwd_options(N):
    M = 45
    dy, r, dres = (rows(M, N, BF, s) for s in (81, 82, 83))
    w, _ = params(N, SF, 84)
    dx, db, dw, dbias = check_bwd(dy, r, w, dres=dres, p=0.3, want_branch=True)
    # the same call again: the same bits
    dx2, db2, dw2, dbias2 = check_bwd(dy, r, w, dres=dres, p=0.3, want_branch=True)
    for a, b in ((dx, dx2), (db, db2), (dw, dw2), (dbias, dbias2)):
        assert torch.equal(a, b)
    mean, rstd = stats(r)
    # accumulation is one float32 addition to what was there
    start = torch.randn(N, generator=gen(1)).cuda()
    _, _, dw3, dbias3 = run_bwd(dy, r, mean, rstd, w, flags=B.ACCUMULATE, dweight=start.clone(), dbias=start.clone())
    assert torch.equal(dw3, start + dw) and torch.equal(dbias3, start + dbias)
    # without the column sums, and with one of them
    dx4 = out_like(M, N, BF)
    B.layer_norm_bwd(dy, r, mean, rstd, w, dx4, dresidual=dres)
    assert torch.equal(dx4, dx)
    ws = torch.empty(B.layer_norm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    only = torch.zeros(N, device="cuda")
    B.layer_norm_bwd(dy, r, mean, rstd, w, dx4, dbias=only, workspace=ws)
    assert torch.equal(only, dbias)
    # no weight: all ones
    check_bwd(dy, r, None, dres=dres)
    # in place: dx over dresidual, dbranch over dy
    a, c = dres.clone(), dy.clone()
    run_bwd(c, r, mean, rstd, w, dres=a, p=0.3, rng=rng_of(1, 2), dx=a, db=c)
    assert torch.equal(a, dx) and torch.equal(c, db)
    # and dx over dy, over r
    a = dy.clone()
    _, _, dw5, dbias5 = run_bwd(a, r, mean, rstd, w, dres=dres, dx=a)
    assert torch.equal(a, dx) and torch.equal(dw5, dw) and torch.equal(dbias5, dbias)
    a = r.clone()
    _, _, dw5, dbias5 = run_bwd(dy, a, mean, rstd, w, dres=dres, dx=a)
    assert torch.equal(a, dx) and torch.equal(dw5, dw) and torch.equal(dbias5, dbias)


@pytest.mark.parametrize("N", [5, 64, 129, 2056])
def test_bwd_against_differences(N):
    """Directional derivatives of the 64-bit forward by central differences.  The second-order
    remainder of a step h along a unit-scale direction is below h^2 times the third derivative (a
    few units of the loss here), and the difference's rounding below 1e-16 |loss| / h."""
    M, h = 6, 1e-4
    rng = np.random.default_rng(N)
    r, dy, dres = (torch.from_numpy(rng.standard_normal((M, N))).float().cuda() for _ in range(3))
    w, b = torch.from_numpy(1 + 0.2 * rng.standard_normal(N)).float().cuda(), torch.zeros(N, device="cuda")
    mean, rstd = stats(r)
    dx, _, dweight, dbias = run_bwd(dy, r, mean, rstd, w, dres=dres)

    def loss(rr, ww, bb):
        return (R.norm_fwd(rr, ww, bb, 1e-5)[0] * f64(dy)).sum() + (f64(dres) * rr).sum()

    r64, w64, b64 = f64(r), f64(w), f64(b)
    for k in range(4):
        for which, grad in ((0, dx), (1, dweight), (2, dbias)):
            base = [r64, w64, b64]
            u = rng.standard_normal(base[which].shape)
            plus, minus = list(base), list(base)
            plus[which], minus[which] = base[which] + h * u, base[which] - h * u
            diff = (loss(*plus) - loss(*minus)) / (2 * h)
            got = (f64(grad) * u).sum()
            size = np.abs(f64(grad) * u).sum() + np.abs(f64(dy)).sum()
            # float32 gradient: 2^-24 times the chain of the sums; statistics given in float32 likewise
            assert abs(got - diff) <= size * (R.row_chain(N) * 4 * R.E + 1e-6), (which, k, got, diff)


@pytest.mark.parametrize("N", [64, 1600, 1001, 33000])
def test_bwd_hard_rows(N):
    """A NaN or an infinity in a row reaches that row's dx and the column sums, no other row."""
    dy, r = rows(9, N, SF, 91), rows(9, N, SF, 92)
    w, _ = params(N, SF, 93)
    mean, rstd = stats(r)
    dx, _, _, dbias = run_bwd(dy, r, mean, rstd, w)
    dy[4, N // 2] = float("nan")
    dx2, _, dw2, dbias2 = run_bwd(dy, r, mean, rstd, w)
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(dx2[keep], dx[keep]) and dx2[4].isnan().all()
    assert dbias2[N // 2].isnan() and dw2[N // 2].isnan() and int(dbias2.isnan().sum()) == 1
    # rstd of a row without deviation: eps alone; dy = 0 gives exactly dresidual
    r[2] = 3.0
    mean, rstd = stats(r)
    dy[4] = 0.0
    dres = rows(9, N, SF, 94)
    dx3, _, _, _ = run_bwd(dy, r, mean, rstd, w, dres=dres)
    assert dx3.isfinite().all() and torch.equal(dx3[4], dres[4])


def test_bwd_many_rows():
    """More rows than any grid has CTAs, and the exactly representable case: dy = 1, xhat = +-1."""
    M, N = 40000, 64
    r = torch.ones(M, N, dtype=BF, device="cuda")
    r[:, ::2] = -1.0
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    dy = torch.ones(M, N, dtype=BF, device="cuda")
    _, _, dw, dbias = run_bwd(dy, r, mean, rstd, None)
    want = torch.full((N,), float(M), device="cuda")
    assert torch.equal(dbias, want)
    want[::2] = -float(M)
    assert torch.equal(dw, want)


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    amax, sat = torch.ones(1, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    B.layer_norm_fwd(x, w, w, x, scale=amax.clone(), amax_out=amax, sat_count=sat)
    assert amax.item() == 0 and sat.item() == 0
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, device="cuda")
    B.layer_norm_bwd(x, x, none, none, w, x, dweight=dw, dbias=db, flags=B.ACCUMULATE)
    assert (dw == 1).all() and (db == 1).all()
    B.layer_norm_bwd(x, x, none, none, w, x, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    B.dropout_fwd(x, x, 0.5, rng_of(1, 1))
    B.dropout_bwd(x, x, 0.5, rng_of(1, 1))


@pytest.mark.parametrize("N,odd", [(1600, 0), (1600, 1)])
def test_offsets_past_32_bits(N, odd):
    """Rows 2^26 (+ 1) elements apart: the last ones start past element 2^32.  The buffer is 10 GB,
    of which the rows alone are written."""
    M, ld = 80, (1 << 26) + 8 + odd
    buf = torch.empty(M * ld, dtype=BF, device="cuda")
    x = torch.as_strided(buf, (M, N), (ld, 1), 0)
    y = torch.as_strided(buf, (M, N), (ld, 1), 1 << 20)
    dx = torch.as_strided(buf, (M, N), (ld, 1), 1 << 21)
    x.copy_(rows(M, N, BF, 5))
    w, b = params(N, SF, 6)
    small = x.contiguous()
    _, mean, rstd = check_fwd(small, w, b)
    y2, mean2, rstd2 = out_like(M, N, BF), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    B.layer_norm_fwd(small, w, b, y2)
    B.layer_norm_fwd(x, w, b, y, mean=mean2, rstd=rstd2)
    tol = R.fwd_tolerances(f64(small), f64(w), f64(b), 1e-5, BF)
    for a, c, t in zip((y, mean2, rstd2), (y2, mean, rstd), tol):
        assert_within(f64(a), f64(c), 2 * t, "forward")
    rng = rng_of(1, 2)
    want = torch.empty_like(small)
    B.dropout_fwd(small, want, 0.5, rng)
    B.dropout_fwd(x, y, 0.5, rng)
    assert torch.equal(y, want)
    dy = rows(M, N, BF, 7)
    y.copy_(dy)
    got = run_bwd(y, x, mean, rstd, w, dx=dx)
    ref = run_bwd(dy, small, mean, rstd, w)
    assert torch.equal(got[0], ref[0])
    tol = R.bwd_tolerances(f64(dy), f64(small), f64(mean), f64(rstd), f64(w), None, BF)
    for a, c, t in zip(got[2:], ref[2:], tol[2:]):  # another alignment may take another order
        assert_within(f64(a), f64(c), 2 * t, "column sums")


def test_side_stream_and_graph():
    """On a stream of its own, and captured: a replay reads the generator state of the moment."""
    M, N = 64, 768
    x, res = rows(M, N, BF, 1), rows(M, N, BF, 2)
    w, b = params(N, SF, 3)
    rng = rng_of(1, 1)
    r, y = out_like(M, N, BF), out_like(M, N, BF)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dy, dx, db = rows(M, N, BF, 4), out_like(M, N, BF), out_like(M, N, BF)
    dw, dbias = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.empty(B.layer_norm_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    amax, q = torch.zeros(1, device="cuda"), torch.empty(M, N, dtype=torch.uint8, device="cuda")
    scale = torch.full((1,), 30.0, device="cuda")

    def step():
        B.layer_norm_fwd(x, w, b, y, mean=mean, rstd=rstd, residual=res, r_out=r, p=0.1, rng=rng, scale=scale, q_out=q,
                         amax_out=amax)
        B.layer_norm_bwd(dy, r, mean, rstd, w, dx, dweight=dw, dbias=dbias, workspace=ws, p=0.1, rng=rng, dbranch=db)
        B.dropout_bwd(dy, y, 0.1, rng)

    outs = (r, y, dx, db, dw, dbias, amax, q)
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng[1] = 5
    g.replay()
    torch.cuda.synchronize()
    keep = R.keep_mask(1, 5, M, N, 0.1)
    assert torch.equal(r.cpu(), R.residual_stream(x.cpu(), res.cpu(), keep, 0.1))
    assert torch.equal((db == 0).cpu() | torch.from_numpy(keep), torch.ones(M, N, dtype=torch.bool))
    rng[1] = 1
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, first))


def test_binding_refusals():
    x = rows(8, 64, BF, 1)
    w = torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    bad = [
        (ValueError, lambda: B.layer_norm_fwd(x, w[:63], w, y)),
        (TypeError, lambda: B.layer_norm_fwd(x, w, w.half(), y)),
        (TypeError, lambda: B.layer_norm_fwd(x, w, w, y.half())),
        (ValueError, lambda: B.layer_norm_fwd(x, w, w, y[:7])),
        (ValueError, lambda: B.layer_norm_fwd(x[:1].expand(8, 64), w, w, y)),
        (ValueError, lambda: B.layer_norm_fwd(x.t(), w[:8], None, torch.empty(64, 8, dtype=BF, device="cuda"))),
        (ValueError, lambda: B.layer_norm_fwd(x, w, w, y, mean=torch.empty(7, device="cuda"))),
        (TypeError, lambda: B.layer_norm_fwd(x, w, w, y, rstd=torch.empty(8, device="cuda", dtype=torch.float64))),
        (ValueError, lambda: B.layer_norm_fwd(x, w, w, y, p=0.5, rng=torch.zeros(1, dtype=torch.int64, device="cuda"))),
        (TypeError, lambda: B.layer_norm_fwd(x, w, w, y, p=0.5, rng=torch.zeros(2, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: B.layer_norm_fwd(x, w, w, y, scale=w[:1], q_out=torch.empty(8, 63, dtype=torch.uint8, device="cuda"))),
        (B.Fp8qError, lambda: B.layer_norm_fwd(x, w, w, y, p=0.5)),
        (B.Fp8qError, lambda: B.layer_norm_fwd(x, w, w, None)),
        (B.Fp8qError, lambda: B.layer_norm_fwd(x, w, w, y, eps=-1.0)),
        (B.Fp8qError, lambda: B.dropout_fwd(x, y, 1.5, rng_of(1, 1))),
        (B.Fp8qError, lambda: B.dropout_fwd(x, y, 0.5, None)),
        (TypeError, lambda: B.dropout_bwd(x, y.float(), 0.5, rng_of(1, 1))),
        (B.Fp8qError, lambda: B.layer_norm_bwd(x, x, w[:8], w[:8], w, y, dweight=w.clone())),
        (B.Fp8qError, lambda: B.layer_norm_bwd(x, x, w[:8], w[:8], w, y, dbias=w.clone(),
                                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: B.layer_norm_bwd(x, x, w[:7], w[:8], w, y)),
        (B.Fp8qError, lambda: B.dropout_bwd(*(2 * [torch.empty(8, 0, dtype=BF, device="cuda")]), 0.5, rng_of(1, 1))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was not refused")
