"""Layer norm and dropout over many more rows than the persistent kernels hold at a time, so that
ring slots, double buffers, carried addresses and prefetched statistics are all used again, and the
last rows are too few for every CTA; each also in place, on and off the 16-byte grid.

The reference is float64 (in torch, by blocks of rows).  r, masks and codes are exact.  The
gradient's column sums are taken from small integers and powers of two, where float32 sums of any
order are exact (below 2^24), so that one row too many, too few or under another row's statistics
shows.  y and dx have the tolerances of norm_reference.py and test_norm_edges_gpu.py."""
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from tests import norm_reference as R
from tests.norm_reference import E
from tests.test_norm_gpu import BF, HF, SF, ids, params, rng_of

pytestmark = pytest.mark.gpu

BLOCK = 1 << 22  # elements of a block of the reference


def blocks(M, N):
    step = max(1, BLOCK // N)
    return [slice(lo, min(M, lo + step)) for lo in range(0, M, step)]


def within(got, want, tol, name):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} outside tolerance, first at {bad.nonzero()[0].tolist()}"


def values(M, N, T, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, N, generator=g, device="cuda").mul_(std).to(T)


def integers(M, N, T, seed, most):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, (M, N), generator=g, device="cuda").to(T)


def stream(x, res, keep, p):
    """r = T(float32(res + (keep ? float32(x * inv) : 0))): separate float32 operations."""
    v = torch.where(keep, x.float() * torch.tensor(1.0 / (1.0 - p), dtype=torch.float32, device="cuda"), torch.zeros((), device="cuda"))
    return (v if res is None else res.float() + v).to(x.dtype)


def mask(seed, off, M, N, p, device="cuda"):
    """norm_reference.keep_mask on the device (int64: the low 64 bits of a product, and its high word masked)."""
    low, quads = 0xFFFFFFFF, (N + 3) // 4
    c = [torch.arange(quads, device=device)[None, :], torch.arange(M, device=device)[:, None],
         torch.tensor(off & low, device=device), torch.tensor(off >> 32, device=device)]
    k = [seed & low, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 & low ^ c[1] ^ k[0], b & low, a >> 32 & low ^ c[3] ^ k[1], a & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return torch.stack([v.expand(M, quads) >= round(p * 2 ** 32) for v in c], 2).reshape(M, 4 * quads)[:, :N]


def check_norm(y, mean, rstd, r, w, b, eps, T):
    """norm_reference.fwd_tolerances, by blocks."""
    N = r.shape[1]
    L = R.row_chain(N)
    for s in blocks(*r.shape):
        x = r[s].double()
        m = x.mean(1)
        d = x - m[:, None]
        rs = ((d * d).mean(1) + eps).rsqrt()
        want = d * rs[:, None] * w + b
        t_mean = (L + 2) * E * x.abs().mean(1)
        rel = (L + 6) * E + t_mean ** 2 * rs ** 2 + 2 * E * d.abs().mean(1) * x.abs().amax(1) * rs ** 2
        t_rstd = rs * (0.5 * rel / (1 - rel).clamp(min=0.5) + 4 * E)
        t = (w.abs() * (rs[:, None] * (t_mean[:, None] + 2 * E * d.abs()) + d.abs() * t_rstd[:, None] * 1.01)
             + 4 * E * ((d * rs[:, None] * w).abs() + b.abs()))
        within(y[s], want, t + R.U[T] * (want.abs() + t) + R.TINY[T], "y")
        within(mean[s], m, t_mean, "mean")
        within(rstd[s], rs, t_rstd, "rstd")


# rows: more than three times what as many CTAs take at a time as the threads of 152 multiprocessors allow
CASES = [(1000003, 7, BF), (250007, 63, BF), (250001, 64, SF), (30011, 768, BF), (30011, 1001, BF), (30011, 1001, SF),
         (20011, 1001, HF), (20011, 1600, BF), (15013, 1601, SF), (8009, 2056, BF), (6007, 4096, SF), (6007, 4099, BF),
         (3001, 4099, SF), (1531, 12345, BF), (1531, 16384, BF), (1021, 12347, SF), (2503, 20000, BF)]


def name(v):
    return ids.get(v) if isinstance(v, torch.dtype) else None


def test_mask_of_this_file():
    args = 0xDEADBEEF12345678, 0xFEDCBA9876543210, 37, 1003, 0.3
    assert torch.equal(mask(*args).cpu(), torch.from_numpy(R.keep_mask(*args)))


@pytest.mark.parametrize("M,N,T", CASES, ids=name)
def test_forward(M, N, T):
    x, res = values(M, N, T, 1), values(M, N, T, 2, 2.0)
    w, b = params(N, SF, 3)
    seed, off, p, eps = 21, 5, 0.2, 1e-5
    rng, keep = rng_of(seed, off), mask(seed, off, M, N, p)
    w64, b64 = w.double(), b.double()

    def call(x, res, y, r_out, **kw):
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        B.layer_norm_fwd(x, w, b, y, eps=eps, mean=mean, rstd=rstd, residual=res, r_out=r_out, **kw)
        return mean, rstd

    y, r = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    mean, rstd = call(x, None, y, None)  # the norm alone
    check_norm(y, mean, rstd, x, w64, b64, eps, T)
    scale = torch.full((1,), 150.0, device="cuda")
    q, amax = torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    sat = torch.zeros(1, dtype=torch.int64, device="cuda")
    codes = dict(fmt=B.E4M3, scale=scale, q_out=q, amax_out=amax, sat_count=sat)
    mean, rstd = call(x, res, y, r, p=p, rng=rng, **codes)  # all of it
    assert torch.equal(r, stream(x, res, keep, p))
    check_norm(y, mean, rstd, r, w64, b64, eps, T)
    v = y.float() * scale
    assert torch.equal(q, B.fp8_cast_f32(v, B.E4M3))
    assert amax.item() == y.float().abs().max().item() and sat.item() == int((v.abs() > 448.0).sum())
    # in place: r over the residual, y over the branch; and without a residual, r over the branch
    x2, res2 = x.clone(), res.clone()
    call(x2, res2, x2, res2, p=p, rng=rng)
    assert torch.equal(x2, y) and torch.equal(res2, r)
    x2, y2 = x.clone(), torch.empty_like(x)
    call(x2, None, y2, x2, p=p, rng=rng)
    assert torch.equal(x2, stream(x, None, keep, p))
    y3 = torch.empty_like(x)
    call(x2, None, y3, None)
    assert torch.equal(y2, y3)


@pytest.mark.parametrize("M,N,T", CASES, ids=name)
def test_backward(M, N, T):
    dy, r, dres = integers(M, N, T, 11, 3), integers(M, N, T, 12, 7), values(M, N, T, 13)
    w, _ = params(N, SF, 14)
    g = torch.Generator(device="cuda").manual_seed(15)
    mean = torch.randint(-3, 4, (M,), generator=g, device="cuda").float()
    rstd = 0.5 * torch.randint(1, 3, (M,), generator=g, device="cuda").float()
    seed, off, p = 31, 6, 0.25
    rng, keep = rng_of(seed, off), mask(seed, off, M, N, p)
    ws = torch.full((B.layer_norm_bwd_workspace_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(dy, r, dres, dx, db, sums=True, **kw):
        dw, dbias = torch.full((N,), 3.0, device="cuda"), torch.full((N,), 3.0, device="cuda")
        cols = dict(dweight=dw, dbias=dbias, workspace=ws) if sums else {}
        B.layer_norm_bwd(dy, r, mean, rstd, w, dx, dresidual=dres, dbranch=db, **cols, **kw)
        return dw, dbias

    dx, db, dx_plain = (torch.full_like(dy, 7.0) for _ in range(3))
    sums = call(dy, r, dres, dx, db, p=p, rng=rng)
    plain_sums = call(dy, r, None, dx_plain, None)
    L, w64, inv = R.row_chain(N), w.double(), 1.0 / (1.0 - p)
    dw, dbias, sizes = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(3))
    for s in blocks(M, N):
        d64, m, rs = dy[s].double(), mean[s, None].double(), rstd[s, None].double()
        xhat = (r[s].double() - m) * rs
        dw += (d64 * xhat).sum(0)
        dbias += d64.sum(0)
        sizes += (d64 * xhat).abs().sum(0)
        g64 = d64 * w64
        c1, c2 = g64.mean(1, keepdim=True), (g64 * xhat).mean(1, keepdim=True)
        t_c1, t_c2 = (L + 4) * E * g64.abs().mean(1, keepdim=True), (L + 7) * E * (g64 * xhat).abs().mean(1, keepdim=True)
        t0 = rs * (t_c1 + xhat.abs() * t_c2 + 3 * E * (xhat * c2).abs() + 2 * E * (g64.abs() + c1.abs() + (xhat * c2).abs()))
        dr0 = rs * (g64 - c1 - xhat * c2)
        dr = dr0 + dres[s].double()
        t = t0 + 2 * E * (dr.abs() + dres[s].double().abs())
        within(dx[s], dr, t + R.U[T] * (dr.abs() + t) + R.TINY[T], "dx")
        k = keep[s]
        within(db[s], torch.where(k, dr * inv, 0.0), inv * t + (R.U[T] + 2 * E) * inv * (dr.abs() + t) + R.TINY[T], "dbranch")
        assert not db[s][~k].any()
        t = t0 + 2 * E * dr0.abs()
        within(dx_plain[s], dr0, t + R.U[T] * (dr0.abs() + t) + R.TINY[T], "dx alone")
    assert sizes.max().item() < 2 ** 23  # multiples of a half: float32 sums of any order are exact
    for got in (sums, plain_sums):
        assert torch.equal(got[0].double(), dw) and torch.equal(got[1].double(), dbias)
    # in place: dx over the residual's gradient, the branch's over dy; dx over r
    a, c = dres.clone(), dy.clone()
    sums2 = call(c, r, a, a, c, p=p, rng=rng)
    assert torch.equal(a, dx) and torch.equal(c, db)
    assert all(torch.equal(u, v) for u, v in zip(sums2, sums))
    a = r.clone()
    call(dy, a, None, a, None)
    assert torch.equal(a, dx_plain)
    a = dy.clone()
    call(a, r, dres, a, None, sums=False)
    assert torch.equal(a, dx)


@pytest.mark.parametrize("T", [BF, HF, SF], ids=ids.get)
@pytest.mark.parametrize("M,N", [(1000003, 7), (200003, 63), (60013, 333), (20011, 1001), (20011, 1601), (30011, 768),
                                 (16387, 1024)])
def test_dropout(M, N, T):
    x, res = values(M, N, T, 41), values(M, N, T, 42, 2.0)
    seed, off, p = 51, 7, 0.3
    rng, keep = rng_of(seed, off), mask(seed, off, M, N, p)
    for residual in (None, res):
        want = stream(x, residual, keep, p)
        y = torch.full_like(x, 7.0)
        B.dropout_fwd(x, y, p, rng, residual=residual)
        assert torch.equal(y, want)
        y = x.clone()  # over the branch
        B.dropout_fwd(y, y, p, rng, residual=residual)
        assert torch.equal(y, want)
        if residual is not None:  # over the residual
            y = residual.clone()
            B.dropout_fwd(x, y, p, rng, residual=y)
            assert torch.equal(y, want)
    y = x.clone()
    B.dropout_bwd(y, y, p, rng)
    assert torch.equal(y, stream(x, None, keep, p))


@pytest.mark.parametrize("T", [HF, SF], ids=ids.get)
@pytest.mark.parametrize("fmt", [B.E4M3, B.E5M2])
@pytest.mark.parametrize("M,N", [(1, 16), (3, 7), (70, 33), (33, 768), (9, 1600), (5, 1001), (3, 4096), (3, 4099),
                                 (2, 12345), (2, 40000)])
def test_codes_of_wider_types(M, N, fmt, T):
    """From float16 and float32 too: the codes, amax and count of the y that the call returns."""
    x = values(M, N, T, 61)
    w, b = params(N, T, 62)
    y = torch.full_like(x, 7.0)
    q = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")
    amax, sat = torch.full((1,), 99.0, device="cuda"), torch.full((1,), 99, dtype=torch.int64, device="cuda")
    scale = torch.full((1,), 300.0 if fmt == B.E4M3 else 40000.0, device="cuda")
    B.layer_norm_fwd(x, w, b, y, fmt=fmt, scale=scale, q_out=q, amax_out=amax, sat_count=sat)
    v = y.float() * scale
    assert torch.equal(q, B.fp8_cast_f32(v, fmt))
    assert amax.item() == y.float().abs().max().item()
    want = int(v.abs().gt(448.0 if fmt == B.E4M3 else 57344.0).sum())
    assert sat.item() == want
    # codes alone, off their own grid, accumulating
    q_off = torch.zeros(M * N + 1, dtype=torch.uint8, device="cuda")[1:].view(M, N)
    B.layer_norm_fwd(x, w, b, None, fmt=fmt, scale=scale, q_out=q_off, amax_out=amax, sat_count=sat, flags=B.ACCUMULATE)
    assert torch.equal(q_off, q) and sat.item() == 2 * want and amax.item() == y.float().abs().max().item()
