"""fp8_glu_fwd and fp8_gemm_dgrad_glu against the 64-bit definition (glu_reference.py).

The GEMM's result is checked within a derived tolerance, and everything that hangs on the rounded
values (codes, their transposes, maximum, saturations) exactly against the BF16 output."""
import pytest
import torch

from tests import glu_reference as R

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def B():
    from quantize_fp8_gemm_gb300 import binding
    return binding


def codes(gen, rows, cols, fmt, most):
    v = torch.randn(rows, cols, generator=gen, device="cuda") * (most / 6)
    return v.clamp(-most, most).to(fmt).view(torch.uint8)


def cell(v):
    return torch.full((1,), float(v), device="cuda")


def fwd_inputs(M, F, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, w = codes(gen, M, K, E4, 224.0), codes(gen, 2 * F, K, E4, 224.0)
    return x, w, cell(224 / 6), cell(224 / 6 * K ** 0.5)


def bwd_inputs(M, F, N, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dy, w = codes(gen, M, N, E5, 28672.0), codes(gen, F, N, E4, 224.0)
    h = torch.randn(M, 2 * F, generator=gen, device="cuda").to(torch.bfloat16)
    return dy, w, cell(28672 / 6), cell(224 / 6 * N ** 0.5), h


def poison(*shape, dtype):
    return torch.full(shape, 0x5A if dtype == torch.uint8 else 7.0, dtype=dtype, device="cuda")


def check_codes(v, scale, fmt, q, q_t, amax, sat):
    want, n = R.codes_of(v, scale, fmt)
    if q is not None:
        assert torch.equal(q, want)
    if q_t is not None:
        assert torch.equal(q_t, want.t())
    assert float(amax) == float(v.abs().max())
    assert int(sat) == n


# one token to several row tiles of pairs, widths of one block to several column tiles, ends inside boxes
SHAPES = [(1, 16, 16), (1, 208, 1600), (1, 48, 8192), (1, 32, 8208), (2, 2000, 528), (3, 16, 64), (4, 10000, 96), (5, 64, 2064), (16, 48, 32), (31, 80, 144), (64, 128, 64), (100, 272, 400),
          (128, 256, 128), (129, 144, 528), (256, 512, 768), (300, 1040, 96), (1000, 336, 256), (2048, 2736, 128)]


@pytest.mark.parametrize("M,F,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(B, M, F, K, act):
    x, w, sx, sw = fwd_inputs(M, F, K, M * 7 + F)
    h, a = poison(M, 2 * F, dtype=torch.bfloat16), poison(M, F, dtype=torch.bfloat16)
    q = poison(M, F, dtype=torch.uint8)
    q_t = poison(F, M, dtype=torch.uint8) if M % 16 == 0 else None
    amax, sat, status = cell(3.0), torch.full((1,), 9, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = cell(300.0)  # saturates the largest products
    B.fp8_glu_fwd(x, w, sx, sw, act=R.ACTS[act], h_out=h, act_out=a, scale_a=s, a_q=q, a_q_t=q_t, amax_out=amax,
                  sat_count=sat, status=status)
    assert int(status) == 0
    g64, u64, a64, tg, tu, ta = R.fwd(x.view(E4).double() / sx.double(), w.view(E4).double() / sw.double(), act)
    R.assert_within(h[:, :F], g64, tg, "g")
    R.assert_within(h[:, F:], u64, tu, "u")
    R.assert_within(a, a64, ta, "a")
    check_codes(a, s, E4, q, q_t, amax, sat)


@pytest.mark.parametrize("act", ["identity", "relu", "relu2"])
@pytest.mark.parametrize("M,F,K", [(48, 80, 144), (272, 400, 128)])
def test_forward_activations(B, M, F, K, act):
    x, w, sx, sw = fwd_inputs(M, F, K, 5)
    a, q, amax, sat = poison(M, F, dtype=torch.bfloat16), poison(M, F, dtype=torch.uint8), cell(0), torch.zeros(1, dtype=torch.int64, device="cuda")
    B.fp8_glu_fwd(x, w, sx, sw, act=R.ACTS[act], act_out=a, scale_a=cell(40), a_q=q, amax_out=amax, sat_count=sat)
    *_, a64, _, _, ta = R.fwd(x.view(E4).double() / sx.double(), w.view(E4).double() / sw.double(), act)
    R.assert_within(a, a64, ta, "a")
    check_codes(a, cell(40), E4, q, None, amax, sat)


@pytest.mark.parametrize("M,F,N", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(B, M, F, N, act):
    dy, w, sdy, sw, h = bwd_inputs(M, F, N, M * 3 + F)
    dh, q = poison(M, 2 * F, dtype=torch.bfloat16), poison(M, 2 * F, dtype=torch.uint8)
    q_t = poison(2 * F, M, dtype=torch.uint8) if M % 16 == 0 else None
    amax, sat, status = cell(3.0), torch.full((1,), 9, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = cell(30000.0)
    B.fp8_gemm_dgrad_glu(dy, w, sdy, sw, h, act=R.ACTS[act], dh=dh, scale_dh=s, dh_q=q, dh_q_t=q_t, amax_out=amax,
                         sat_count=sat, status=status)
    assert int(status) == 0
    want, tol = R.bwd(dy.view(E5).double() / sdy.double(), w.view(E4).double() / sw.double(), h.double(), act)
    R.assert_within(dh, want, tol, "dh")
    check_codes(dh, s, E5, q, q_t, amax, sat)


@pytest.mark.parametrize("act", ["identity", "relu", "relu2"])
@pytest.mark.parametrize("M,F,N", [(48, 80, 144), (272, 400, 128)])
def test_backward_activations(B, M, F, N, act):
    dy, w, sdy, sw, h = bwd_inputs(M, F, N, 6)
    dh = poison(M, 2 * F, dtype=torch.bfloat16)
    B.fp8_gemm_dgrad_glu(dy, w, sdy, sw, h, act=R.ACTS[act], dh=dh)
    want, tol = R.bwd(dy.view(E5).double() / sdy.double(), w.view(E4).double() / sw.double(), h.double(), act)
    R.assert_within(dh, want, tol, "dh")


TILES = [(0, 64), (0, 128), (0, 192), (0, 256), (1, 128), (1, 192), (1, 256)]


@pytest.fixture
def tile(B, request):
    B.fp8q_glu_set_tile(*request.param)
    yield request.param
    B.fp8q_glu_set_tile(-1)


@pytest.mark.parametrize("M,F,K", [(144, 272, 80), (496, 1040, 336), (4000, 144, 48)])
@pytest.mark.parametrize("tile", TILES, indirect=True, ids=str)
def test_every_tile(B, tile, M, F, K):
    """Each tile at ends inside its rows, chunks and 128-byte k-blocks; results do not depend on it."""
    test_forward(B, M, F, K, "silu")
    test_backward(B, M, F, K, "gelu")
    x, w, sx, sw = fwd_inputs(M, F, K, 5)
    a, b = poison(M, F, dtype=torch.bfloat16), poison(M, F, dtype=torch.bfloat16)
    B.fp8_glu_fwd(x, w, sx, sw, act_out=a)
    B.fp8q_glu_set_tile(-1)
    B.fp8_glu_fwd(x, w, sx, sw, act_out=b)
    assert torch.equal(a, b)


def test_tile_hook_refuses(B):
    for bad in ((0, 96), (1, 64), (2, 128), (0, 0)):
        with pytest.raises(B.Fp8qError):
            B.fp8q_glu_set_tile(*bad)


@pytest.mark.parametrize("M,F,K", [(48, 80, 144), (272, 400, 128)])
def test_outputs_alone(B, M, F, K):
    """Each optional output asked for by itself has the bits it has among the others."""
    x, w, sx, sw = fwd_inputs(M, F, K, 11)
    bf, u8 = torch.bfloat16, torch.uint8
    h, a, q, q_t = poison(M, 2 * F, dtype=bf), poison(M, F, dtype=bf), poison(M, F, dtype=u8), poison(F, M, dtype=u8)
    B.fp8_glu_fwd(x, w, sx, sw, h_out=h, act_out=a, scale_a=cell(30), a_q=q, a_q_t=q_t)
    for name, full in (("act_out", a), ("a_q", q), ("a_q_t", q_t)):
        one = torch.empty_like(full)
        B.fp8_glu_fwd(x, w, sx, sw, scale_a=cell(30), **{name: one})
        assert torch.equal(one, full), name
    dy, w2, sdy, sw2, hb = bwd_inputs(M, F, K, 12)
    dh, q, q_t = poison(M, 2 * F, dtype=bf), poison(M, 2 * F, dtype=u8), poison(2 * F, M, dtype=u8)
    B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, hb, dh=dh, scale_dh=cell(100), dh_q=q, dh_q_t=q_t)
    for name, full in (("dh", dh), ("dh_q", q), ("dh_q_t", q_t)):
        one = torch.empty_like(full)
        B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, hb, scale_dh=cell(100), **{name: one})
        assert torch.equal(one, full), name
    B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, hb, dh=hb)  # over its input
    assert torch.equal(hb, dh)


@pytest.mark.parametrize("M,F,K", [(48, 64, 48), (272, 208, 64)])
def test_tensors_off_the_32_byte_grid(B, M, F, K):
    """16-byte alignment is all that is asked of a tensor: outputs and h at odd multiples of it."""
    def at16(rows, cols, dtype):
        buf = torch.zeros(rows * cols * dtype.itemsize + 48, dtype=torch.uint8, device="cuda")
        start = 16 if buf.data_ptr() % 32 == 0 else 0
        t = buf[start:start + rows * cols * dtype.itemsize].view(dtype).view(rows, cols)
        assert t.data_ptr() % 32 == 16
        return t, lambda: not buf[:start].any() and not buf[start + rows * cols * dtype.itemsize:].any()

    bf, u8 = torch.bfloat16, torch.uint8
    x, w, sx, sw = fwd_inputs(M, F, K, 21)
    want = [torch.empty(M, 2 * F, dtype=bf, device="cuda"), torch.empty(M, F, dtype=bf, device="cuda"),
            torch.empty(M, F, dtype=u8, device="cuda"), torch.empty(F, M, dtype=u8, device="cuda")]
    outs = [at16(M, 2 * F, bf), at16(M, F, bf), at16(M, F, u8), at16(F, M, u8)]
    for h, a, q, t in (want, [o for o, _ in outs]):
        B.fp8_glu_fwd(x, w, sx, sw, h_out=h, act_out=a, scale_a=cell(30), a_q=q, a_q_t=t)
    assert all(torch.equal(o, v) and clean() for (o, clean), v in zip(outs, want))
    dy, w2, sdy, sw2, hb = bwd_inputs(M, F, K, 22)
    h16 = at16(M, 2 * F, bf)[0]
    h16.copy_(hb)
    want = [torch.empty(M, 2 * F, dtype=bf, device="cuda"), torch.empty(M, 2 * F, dtype=u8, device="cuda"), torch.empty(2 * F, M, dtype=u8, device="cuda")]
    outs = [at16(M, 2 * F, bf), at16(M, 2 * F, u8), at16(2 * F, M, u8)]
    for h, (dh, q, t) in ((hb, want), (h16, [o for o, _ in outs])):
        B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, h, dh=dh, scale_dh=cell(100), dh_q=q, dh_q_t=t)
    assert all(torch.equal(o, v) and clean() for (o, clean), v in zip(outs, want))


def test_large_values_and_gate_tails(B):
    """Gates far in the exponential's tails (it overflows at -89) and squares past float32's range of codes."""
    M, F, N = 32, 64, 48
    dy, w, sdy, sw, h = bwd_inputs(M, F, N, 31)
    g = torch.tensor([-300.0, -100.0, -89.0, -88.0, -30.0, -1e-3, 0.0, 1e-30, 20.0, 88.0, 100.0, 3000.0], device="cuda")
    h[:, :12] = g.to(torch.bfloat16)
    for act in ("silu", "gelu"):
        dh = poison(M, 2 * F, dtype=torch.bfloat16)
        B.fp8_gemm_dgrad_glu(dy, w, sdy, sw, h, act=R.ACTS[act], dh=dh)
        want, tol = R.bwd(dy.view(E5).double() / sdy.double(), w.view(E4).double() / sw.double(), h.double(), act)
        assert bool(torch.isfinite(dh).all())
        R.assert_within(dh, want, tol, act)
    x, w, sx, sw = fwd_inputs(M, F, N, 32)
    for act in ("silu", "gelu"):  # g and u of some thousands, both signs
        a = poison(M, F, dtype=torch.bfloat16)
        B.fp8_glu_fwd(x, w, sx, sw / 3000, act=R.ACTS[act], act_out=a)
        *_, a64, _, _, ta = R.fwd(x.view(E4).double() / sx.double(), w.view(E4).double() / (sw / 3000).double(), act)
        R.assert_within(a, a64, ta, act)


def test_accumulate_and_empty(B):
    x, w, sx, sw = fwd_inputs(32, 48, 64, 3)
    a, amax, sat = poison(32, 48, dtype=torch.bfloat16), cell(1e4), torch.full((1,), 5, device="cuda")
    B.fp8_glu_fwd(x, w, sx, sw, act_out=a, scale_a=cell(1e9), amax_out=amax, sat_count=sat, flags=B.ACCUMULATE)
    assert float(amax) == 1e4 and int(sat) == 5 + R.codes_of(a, cell(1e9), E4)[1]
    none = torch.empty(0, 64, dtype=torch.uint8, device="cuda")
    B.fp8_glu_fwd(none, w, sx, sw, scale_a=cell(1), a_q=none.new_empty(0, 48), amax_out=amax, sat_count=sat)
    assert float(amax) == 0 and int(sat) == 0
    B.fp8_gemm_dgrad_glu(none, w[:48], sx, sw, torch.empty(0, 96, dtype=torch.bfloat16, device="cuda"),
                         dh=torch.empty(0, 96, dtype=torch.bfloat16, device="cuda"), amax_out=cell(2))


def test_infinities_and_nan_stay_in_their_rows(B):
    """A NaN code makes its own row NaN and the maximum with it; the other rows keep their bits.  The
    columns behind F (of the gate's last tile, which reads the up-projection's first rows) count nowhere."""
    M, F, K = 40, 80, 64
    x, w, sx, sw = fwd_inputs(M, F, K, 4)
    a, amax = poison(M, F, dtype=torch.bfloat16), cell(0)
    B.fp8_glu_fwd(x, w, sx, sw, act_out=a, amax_out=amax)
    x2 = x.clone()
    x2[7, 3] = 0x7F  # E4M3 NaN
    b = poison(M, F, dtype=torch.bfloat16)
    B.fp8_glu_fwd(x2, w, sx, sw, act_out=b, amax_out=amax)
    assert bool(torch.isnan(b[7]).all()) and bool(torch.isnan(amax).all())
    keep = torch.arange(M, device="cuda") != 7
    assert torch.equal(a[keep], b[keep])
    # NaN in the up-projection's first rows, which the gate's ragged last box reads too
    w2 = w.clone()
    w2[F + 1, 0] = 0x7F
    B.fp8_glu_fwd(x, w2, sx, sw, act_out=b)
    cols = torch.arange(F, device="cuda") != 1
    assert torch.equal(a[:, cols], b[:, cols]) and bool(torch.isnan(b[:, 1]).all())


def test_captured_and_streams(B):
    M, F, K = 256, 272, 160
    x, w, sx, sw = fwd_inputs(M, F, K, 8)
    ref, amax = poison(M, F, dtype=torch.uint8), cell(0)
    B.fp8_glu_fwd(x, w, sx, sw, scale_a=cell(30), a_q=ref, amax_out=amax)
    got, amax2, s = torch.empty_like(ref), cell(0), cell(30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.fp8_glu_fwd(x, w, sx, sw, scale_a=s, a_q=got, amax_out=amax2)
    side.synchronize()
    assert torch.equal(got, ref) and torch.equal(amax, amax2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.fp8_glu_fwd(x, w, sx, sw, scale_a=s, a_q=got, amax_out=amax2)
    x.copy_(x.flip(0))
    for _ in range(3):
        got.zero_()
        amax2.fill_(1e9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref.flip(0)) and torch.equal(amax, amax2)


@pytest.mark.parametrize("M", [64, 300])
def test_a_wait_that_runs_out_is_reported(B, M):
    """No operand arrives (a hook): the kernels give up after about 2 s, say so and leave the context usable."""
    F, K = 80, 64
    x, w, sx, sw = fwd_inputs(M, F, K, 8)
    dy, w2, sdy, sw2, h = bwd_inputs(M, F, K, 9)
    a, dh = poison(M, F, dtype=torch.bfloat16), poison(M, 2 * F, dtype=torch.bfloat16)
    want = [t.clone() for t in (a, dh)]
    B.fp8_glu_fwd(x, w, sx, sw, act_out=want[0])
    B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, h, dh=want[1])
    for call in (lambda st: B.fp8_glu_fwd(x, w, sx, sw, act_out=a, status=st), lambda st: B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, h, dh=dh, status=st)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.fp8q_gemm_test_hold_loads(True)
        try:
            call(status)
            torch.cuda.synchronize()
        finally:
            B.fp8q_gemm_test_hold_loads(False)
        assert int(status) & B.DEV_TIMEOUT
        status.zero_()
        call(status)
        assert int(status) == 0
    assert torch.equal(a, want[0]) and torch.equal(dh, want[1])


def test_two_streams_at_once(B):
    """Calls of both kernels side by side on two streams have the bits they have alone."""
    M, F, K = 2048, 1040, 256
    sets = [fwd_inputs(M, F, K, 40 + i) for i in range(2)]
    backs = [bwd_inputs(M, F, K, 50 + i) for i in range(2)]

    def run(i, out):
        x, w, sx, sw = sets[i]
        dy, w2, sdy, sw2, h = backs[i]
        for _ in range(4):
            B.fp8_glu_fwd(x, w, sx, sw, scale_a=out[4], a_q=out[0], a_q_t=out[1], amax_out=out[2])
            B.fp8_gemm_dgrad_glu(dy, w2, sdy, sw2, h, dh=out[3])

    def outs():
        return [poison(M, F, dtype=torch.uint8), poison(F, M, dtype=torch.uint8), cell(0), poison(M, 2 * F, dtype=torch.bfloat16), cell(30)]

    alone, both = [outs() for _ in range(2)], [outs() for _ in range(2)]
    for i in range(2):
        run(i, alone[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            run(i, both[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(alone, both) for a, b in zip(x, y))
