"""block_norm_fwd and block_norm_bwd against the 64-bit definition (block_norm_reference.py): types, widths
from one column to beyond the one-pass kernels, rows on and off the 16-byte grid, every optional part."""
import itertools

import pytest
import torch

from tests import block_norm_reference as R

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


def make(M, N, T, seed, pad=0, offset=0, params=FP, gate=False, alpha=False, residual=True):
    """Inputs of one call; [M,N] tensors are cut out of buffers `pad` wider, from column `offset`."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def rows(std):
        return (normal(M, N + pad + offset) * std).to(T)[:, offset:offset + N]

    return dict(x=rows(0.7), residual=rows(2.0) if residual else None, r=rows(2.0), dy=rows(0.5), dr=rows(0.5),
                w=(1 + 0.1 * normal(N)).to(params), wp=(0.3 + 0.05 * normal(N)).to(params),
                gate=normal(M).sigmoid() if gate else None, alpha=torch.full((1,), 0.9, device="cuda") if alpha else None)


def out_like(M, N, T, pad=0, offset=0):
    """An output cut out of a buffer of poison, and a check that the rest of the buffer keeps it."""
    whole = torch.full((M, N + pad + offset), 7.0, dtype=T, device="cuda")

    def untouched():
        return bool((whole[:, :offset] == 7).all()) and bool((whole[:, offset + N:] == 7).all())

    return whole[:, offset:offset + N], untouched


def f64(t):
    return None if t is None else t.double()


def check_fwd(B, M, N, T, post=True, pre=True, pad=0, offset=0, codes=False, fmt=0, **kw):
    s = make(M, N, T, M * 31 + N, pad, offset, **kw)
    r, r_ok = out_like(M, N, T, pad, offset)
    y, y_ok = out_like(M, N, T, pad, offset)
    rstd, rp = torch.full((M,), 5.0, device="cuda"), torch.full((M,), 5.0, device="cuda")
    q = torch.full((M, N), 0x5A, dtype=torch.uint8, device="cuda")
    scale, amax, sat = torch.full((1,), 150.0, device="cuda"), torch.full((1,), 1e9, device="cuda"), torch.full((1,), 3, device="cuda")
    more = dict(fmt=fmt, scale=scale, q_out=q, amax_out=amax, sat_count=sat) if codes else {}
    B.block_norm_fwd(s["x"], s["w"] if pre else None, y if pre else None, eps=EPS, rstd=rstd if pre else None, residual=s["residual"],
                     alpha=s["alpha"], gate=s["gate"], post_weight=s["wp"], post_norm=post,
                     rstd_post=rp if post else None, r_out=r, **more)
    assert r_ok() and y_ok()
    gate = f64(s["gate"]) if s["gate"] is not None else torch.ones(M, dtype=torch.float64, device="cuda")
    alpha = float(s["alpha"]) if s["alpha"] is not None else 1.0
    want, wrp, tr, trp = R.stream(f64(s["x"]), f64(s["residual"]), f64(s["wp"]), gate, alpha, post, EPS)
    R.assert_within(r, want, R.rounded(want, tr, T), "r")
    if post:
        R.assert_within(rp, wrp, trp, "rstd_post")
    if not pre:
        return
    wy, wrstd, ty, trstd = R.norm(f64(r), f64(s["w"]), EPS)
    R.assert_within(rstd, wrstd, trstd, "rstd")
    R.assert_within(y, wy, R.rounded(wy, ty, T), "y")
    if codes:
        ft, most = (torch.float8_e4m3fn, 448.0) if fmt == 0 else (torch.float8_e5m2, 57344.0)
        v = y.float() * scale
        assert torch.equal(q, v.clamp(-most, most).to(ft).view(torch.uint8))
        assert float(amax) == float(y.float().abs().max()) and int(sat) == int((v.abs() > most).sum())


WIDTHS = [1, 3, 8, 12, 64, 100, 250, 256, 264, 512, 520, 768, 1001, 1237, 1600, 2048, 2056, 4099, 4104, 8192, 8200, 16384, 20001]


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("T", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
def test_forward_widths(B, N, T):
    check_fwd(B, 5, N, T, codes=True, gate=True, alpha=True, params=T if N % 3 == 0 else FP)


@pytest.mark.parametrize("post,pre,gate,alpha,residual", list(itertools.product([0, 1], repeat=5)))
def test_forward_parts(B, post, pre, gate, alpha, residual):
    check_fwd(B, 19, 200, BF, post=bool(post), pre=bool(pre), gate=bool(gate), alpha=bool(alpha), residual=bool(residual))
    check_fwd(B, 19, 203, HF, post=bool(post), pre=bool(pre), gate=bool(gate), alpha=bool(alpha), residual=bool(residual))


@pytest.mark.parametrize("M,N,T,pad,offset", [(1, 1600, BF, 0, 0), (1, 16, BF, 0, 0), (33, 64, BF, 8, 0), (40, 333, HF, 3, 1),
                                              (9, 1001, BF, 6, 1), (7, 2500, FP, 1, 3), (4000, 64, BF, 0, 0), (6000, 72, BF, 3, 0),
                                              (3001, 768, BF, 0, 0), (2503, 1600, BF, 16, 8), (1999, 1237, FP, 0, 0), (700, 5000, BF, 0, 0),
                                              (20000, 20, HF, 0, 0), (5003, 1001, HF, 6, 0)])
def test_forward_rows(B, M, N, T, pad, offset):
    """One row to several rounds of the persistent CTAs, rows in wider buffers, starts off the grid."""
    check_fwd(B, M, N, T, pad=pad, offset=offset, codes=True, gate=M % 2 == 1)


def test_forward_e5m2_and_plain_norm(B):
    check_fwd(B, 37, 320, BF, codes=True, fmt=1)
    x = torch.randn(37, 320, device="cuda").to(BF)
    y, y2, r = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    B.block_norm_fwd(x, None, y, eps=EPS, r_out=r)  # the norm before the first block: r is x
    assert torch.equal(r, x)
    B.block_norm_fwd(x, torch.ones(320, device="cuda"), y2, eps=EPS, residual=torch.zeros_like(x))
    assert torch.equal(y, y2)


def bwd_args(s, T, M, N, post, pre, dres, dx, block, sums, rstd, rp):
    return dict(dr=s["dr"], x=s["x"] if block else None, residual=s["residual"] if s["alpha"] is not None else None, alpha=s["alpha"],
                gate=s["gate"], post_weight=s["wp"], post_norm=post, rstd_post=rp, dresidual=dres, dx=dx, **sums)


def check_bwd(B, M, N, T, post=True, pre=True, block=True, with_dr=True, pad=0, offset=0, fill=7.0, flags=0, **kw):
    s = make(M, N, T, M * 17 + N, pad, offset, **kw)
    if not with_dr:
        s["dr"] = None
    dres, ok1 = out_like(M, N, T, pad, offset)
    dx, ok2 = out_like(M, N, T, pad, offset)
    rstd = (s["r"].float().square().mean(1) + EPS).rsqrt() if pre else None
    rp = (s["x"].float().square().mean(1) + EPS).rsqrt() if post else None
    f = lambda n: torch.full((n,), fill, device="cuda")  # noqa: E731
    sums = {}
    if pre:
        sums["dweight"] = f(N)
    if block:
        sums["dpost_weight"] = f(N)
        if s["gate"] is not None:
            sums["dgate"] = f(M)
    if s["alpha"] is not None:
        sums["dalpha"] = f(1)
    ws = torch.full((B.block_norm_bwd_workspace_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")
    B.block_norm_bwd(s["dy"] if pre else None, s["r"] if pre else None, rstd, s["w"] if pre else None, workspace=ws, flags=flags,
                     **bwd_args(s, T, M, N, post, pre, dres, dx if block else None, block, sums, rstd, rp))
    assert ok1() and ok2()
    gate = f64(s["gate"]) if s["gate"] is not None else torch.ones(M, dtype=torch.float64, device="cuda")
    alpha = float(s["alpha"]) if s["alpha"] is not None else 1.0
    want = R.bwd(f64(s["dy"]) if pre else None, f64(s["r"]), f64(rstd), f64(s["w"]), f64(s["dr"]), f64(s["x"]), f64(rp), f64(s["wp"]),
                 gate, alpha, f64(s["residual"]) if s["alpha"] is not None else None, post)
    v, t = want["dresidual"]
    R.assert_within(dres, v, R.rounded(v, t, T), "dresidual")
    if block:
        v, t = want["dx"]
        R.assert_within(dx, v, R.rounded(v, t, T), "dx")
    for name, got in sums.items():
        v, t = want[name]
        if flags and name != "dgate":
            v, t = v + fill, t + R.E * (v + fill).abs()
        R.assert_within(got, v, t, name)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("T", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
def test_backward_widths(B, N, T):
    check_bwd(B, 5, N, T, gate=True, alpha=True, params=T if N % 3 == 0 else FP)
    check_bwd(B, 5, N, T)


@pytest.mark.parametrize("post,pre,block,gate,alpha", list(itertools.product([0, 1], repeat=5)))
def test_backward_parts(B, post, pre, block, gate, alpha):
    for N, T in ((200, BF), (203, HF), (1600, BF)):
        check_bwd(B, 19, N, T, post=bool(post), pre=bool(pre), block=bool(block), gate=bool(gate), alpha=bool(alpha))
        if pre:
            check_bwd(B, 19, N, T, post=bool(post), block=bool(block), with_dr=False, gate=bool(gate), alpha=bool(alpha))


@pytest.mark.parametrize("M,N,T,pad,offset", [(1, 1600, BF, 0, 0), (1, 16, BF, 0, 0), (33, 64, BF, 8, 0), (40, 333, HF, 3, 1),
                                              (9, 1001, BF, 6, 1), (7, 2500, FP, 1, 3), (4000, 64, BF, 0, 0), (6000, 72, BF, 3, 0),
                                              (3001, 768, BF, 0, 0), (2503, 1600, BF, 16, 8), (2999, 1237, FP, 0, 0), (700, 5000, BF, 0, 0),
                                              (20000, 20, HF, 0, 0), (5003, 1001, HF, 6, 0), (2000, 16384, BF, 0, 0)])
def test_backward_rows(B, M, N, T, pad, offset):
    check_bwd(B, M, N, T, pad=pad, offset=offset, gate=M % 2 == 1, alpha=M % 3 == 0)


def test_backward_accumulates_and_repeats(B):
    check_bwd(B, 300, 264, BF, gate=True, alpha=True, flags=B.ACCUMULATE)
    s = make(3000, 1600, BF, 5, alpha=True)
    rstd, rp = (s["r"].float().square().mean(1) + EPS).rsqrt(), (s["x"].float().square().mean(1) + EPS).rsqrt()
    ws = torch.empty(B.block_norm_bwd_workspace_bytes(3000, 1600), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(3):
        sums = dict(dweight=torch.empty(1600, device="cuda"), dpost_weight=torch.empty(1600, device="cuda"), dalpha=torch.empty(1, device="cuda"))
        ws.random_()
        B.block_norm_bwd(s["dy"], s["r"], rstd, s["w"], dr=s["dr"], x=s["x"], residual=s["residual"], alpha=s["alpha"],
                         post_weight=s["wp"], post_norm=True, rstd_post=rp, workspace=ws, **sums)
        got.append(sums)
    for g in got[1:]:
        assert all(torch.equal(g[k], got[0][k]) for k in g)


def test_no_rows(B):
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    amax, sat = torch.ones(1, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    B.block_norm_fwd(e, None, e, scale=amax.clone(), amax_out=amax, sat_count=sat)
    assert float(amax) == 0 and int(sat) == 0
    dw = torch.ones(64, device="cuda")
    B.block_norm_bwd(e, e, torch.empty(0, device="cuda"), None, dr=e, dresidual=e, dweight=dw)
    assert not dw.any()
    dw.fill_(2)
    B.block_norm_bwd(e, e, torch.empty(0, device="cuda"), None, dr=e, dresidual=e, dweight=dw, flags=B.ACCUMULATE)
    assert bool((dw == 2).all())


@pytest.mark.parametrize("M,N,T", [(700, 1600, BF), (700, 1001, HF), (11, 20001, BF), (900, 72, FP), (300, 4104, BF)])
def test_outputs_over_inputs(B, M, N, T):
    s = make(M, N, T, 3)
    r, y = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    kw = dict(eps=EPS, post_weight=s["wp"], post_norm=True)
    B.block_norm_fwd(s["x"], s["w"], y, residual=s["residual"], r_out=r, **kw)
    x, res = s["x"].clone(), s["residual"].clone()
    B.block_norm_fwd(x, s["w"], x, residual=res, r_out=res, **kw)
    assert torch.equal(x, y) and torch.equal(res, r)
    rstd, rp = (s["r"].float().square().mean(1) + EPS).rsqrt(), (s["x"].float().square().mean(1) + EPS).rsqrt()
    dres, dx = torch.empty_like(r), torch.empty_like(r)
    kw = dict(post_weight=s["wp"], post_norm=True, rstd_post=rp)
    B.block_norm_bwd(s["dy"], s["r"], rstd, s["w"], dr=s["dr"], x=s["x"], dresidual=dres, dx=dx, **kw)
    dy, dr = s["dy"].clone(), s["dr"].clone()
    B.block_norm_bwd(dy, s["r"], rstd, s["w"], dr=dr, x=s["x"], dresidual=dr, dx=dy, **kw)
    assert torch.equal(dy, dx) and torch.equal(dr, dres)


def test_infinities_stay_in_their_rows(B):
    for N, T in ((64, BF), (1600, BF), (203, HF), (4104, BF)):
        s = make(40, N, T, 9)
        y, y2 = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        kw = dict(eps=EPS, residual=s["residual"], post_weight=s["wp"], post_norm=True)
        amax = torch.zeros(1, device="cuda")
        B.block_norm_fwd(s["x"], s["w"], y, **kw)
        s["x"][3, N // 2], s["x"][17, 0], s["residual"][30, N - 1] = float("nan"), float("inf"), float("nan")
        B.block_norm_fwd(s["x"], s["w"], y2, scale=torch.ones(1, device="cuda"), amax_out=amax, **kw)
        keep = torch.ones(40, dtype=torch.bool, device="cuda")
        keep[[3, 17, 30]] = False
        assert torch.equal(y[keep], y2[keep])
        assert bool(torch.isnan(y2[3]).all()) and bool(torch.isnan(y2[30]).all()) and bool(torch.isnan(amax).all())


def test_long_rows_past_32_bits(B):
    """Rows whose offsets pass 2^31 elements."""
    M, N = 9, 64
    big = torch.empty((1 << 31) + (1 << 20), dtype=BF, device="cuda")
    ld = (1 << 31) // 8
    x = torch.as_strided(big, (M, N), (ld, 1))
    src = torch.randn(M, N, device="cuda").to(BF)
    x.copy_(src)
    y, want = torch.empty_like(src), torch.empty_like(src)
    B.block_norm_fwd(x, None, y, eps=EPS, r_out=x)
    B.block_norm_fwd(src, None, want, eps=EPS)
    assert torch.equal(y, want) and torch.equal(x, src)


def test_captured(B):
    s = make(1000, 768, BF, 6)
    y, amax, sat = torch.empty_like(s["x"]), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    dw, dx = torch.empty(768, device="cuda"), torch.empty_like(y)
    r, rstd, rp = torch.empty_like(y), torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
    scale = torch.full((1,), 10.0, device="cuda")
    ws = torch.empty(B.block_norm_bwd_workspace_bytes(1000, 768), dtype=torch.uint8, device="cuda")

    def step():
        B.block_norm_fwd(s["x"], s["w"], y, eps=EPS, rstd=rstd, residual=s["residual"], post_weight=s["wp"], post_norm=True,
                         rstd_post=rp, r_out=r, scale=scale, amax_out=amax, sat_count=sat)
        B.block_norm_bwd(s["dy"], r, rstd, s["w"], dr=s["dr"], x=s["x"], post_weight=s["wp"], post_norm=True, rstd_post=rp, dx=dx,
                         dweight=dw, workspace=ws)

    step()
    want = [t.clone() for t in (y, amax, dx, dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (y, dx, dw):
            t.zero_()
        amax.fill_(1e6)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, amax, dx, dw), want))


@pytest.mark.parametrize("N,T", [(64, BF), (250, HF), (1600, BF), (1001, HF), (4104, BF), (20001, BF), (768, FP)])
def test_one_row_and_codes(B, N, T):
    """One row is one CTA, which stores the maximum and count itself; with ACCUMULATE it adds to them."""
    s = make(1, N, T, 77)
    y, q = torch.empty_like(s["x"]), torch.empty(1, N, dtype=torch.uint8, device="cuda")
    amax, sat, scale = torch.full((1,), 1e9, device="cuda"), torch.full((1,), 50, device="cuda"), torch.full((1,), 400.0, device="cuda")
    kw = dict(eps=EPS, residual=s["residual"], post_weight=s["wp"], post_norm=True, scale=scale, q_out=q, sat_count=sat)
    B.block_norm_fwd(s["x"], s["w"], y, amax_out=amax, **kw)
    count = int(((y.float() * 400).abs() > 448).sum())
    assert float(amax) == float(y.float().abs().max()) and int(sat) == count > 0
    big = torch.full((1,), 1e9, device="cuda")
    B.block_norm_fwd(s["x"], s["w"], y, amax_out=big, flags=B.ACCUMULATE, **kw)
    assert float(big) == 1e9 and int(sat) == 2 * count


def test_two_streams_at_once(B):
    """Backward calls side by side, each with a workspace of its own."""
    sets = [make(3000, 1600, BF, 60 + i) for i in range(2)]
    stats = [((s["r"].float().square().mean(1) + EPS).rsqrt(), (s["x"].float().square().mean(1) + EPS).rsqrt()) for s in sets]
    size = B.block_norm_bwd_workspace_bytes(3000, 1600)

    def outs():
        return [torch.empty_like(sets[0]["x"]), torch.empty(1600, device="cuda"), torch.empty(1600, device="cuda"),
                torch.empty(size, dtype=torch.uint8, device="cuda")]

    def run(i, o):
        s, (rstd, rp) = sets[i], stats[i]
        for _ in range(3):
            B.block_norm_bwd(s["dy"], s["r"], rstd, s["w"], dr=s["dr"], x=s["x"], post_weight=s["wp"], post_norm=True, rstd_post=rp,
                             dx=o[0], dweight=o[1], dpost_weight=o[2], workspace=o[3])

    alone, both = [outs() for _ in range(2)], [outs() for _ in range(2)]
    for i in range(2):
        run(i, alone[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            run(i, both[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(alone, both) for a, b in zip(x[:3], y[:3]))


@pytest.mark.parametrize("N,T", [(12288, BF), (16377, HF), (6000, FP), (40000, BF)])
def test_rows_over_a_cluster(B, N, T):
    """Rows that two, four and eight CTAs share, several a cluster."""
    check_bwd(B, 400, N, T, gate=True, alpha=True)
    check_bwd(B, 400, N, T)


@pytest.mark.parametrize("T", [BF, HF, FP], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N", [8, 99, 333, 768, 1001, 1600, 1601, 5001])
def test_infinite_scales_leave_the_statistic_zero(B, N, T):
    """A row under an infinite gate, and every row under an infinite alpha, is infinite, so its statistic is
    exactly 0: columns that lanes have behind the row (0 times an infinity) must not reach its sum."""
    M = 37
    s = make(M, N, T, 1234 + N, gate=True)
    for k in ("x", "residual", "wp"):  # no zeros: 0 times an infinity is NaN in the row itself
        s[k] = torch.where(s[k] == 0, torch.ones_like(s[k]), s[k])
    s["gate"][5] = float("inf")
    y, r = torch.empty(M, N, dtype=T, device="cuda"), torch.empty(M, N, dtype=T, device="cuda")
    rstd = torch.full((M,), 5.0, device="cuda")

    def run(alpha):
        B.block_norm_fwd(s["x"], s["w"], y, eps=EPS, rstd=rstd, residual=s["residual"], alpha=alpha, gate=s["gate"],
                         post_weight=s["wp"], post_norm=True, rstd_post=torch.empty(M, device="cuda"), r_out=r)

    run(None)
    others = [i for i in range(M) if i != 5]
    assert bool(torch.isinf(r[5]).all()) and float(rstd[5]) == 0.0
    assert bool(torch.isfinite(y[others]).all()) and bool((rstd[others] > 0).all())
    s["gate"][5] = 0.5
    run(torch.full((1,), float("inf"), device="cuda"))
    assert bool(torch.isinf(r).all()) and bool((rstd == 0).all())
