"""The gated block's kernels and its norms together, as a training step uses them (Fp8GatedMlpStack).

Each pass is checked against its own 64-bit reference from the tensors that the step fed it, and the
stack as a whole against the float64 model of the same weights.  The second check's bound: an operand in
E4M3 is off by 2.7 % RMS, in E5M2 by twice that, independently per element, so a product of two E4M3
operands by 3.8 %, of an E4M3 and an E5M2 one by 6 %.  The branch has the two projections, whose product
adds them up to at most sqrt(2) 3.8 % (times the activation's slope, at most 1.1), and the
down-projection: sqrt(5.9^2 + 3.8^2) = 7 %.  A gradient passes two products more, and the activation's
derivatives with the error of h: sqrt(7^2 + 6^2 + 6^2 + 3.8^2) = 12 %; one sub-layer above adds its own.
0.12 and 0.25 leave room for the sampling of the errors."""
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from quantize_fp8_gemm_gb300.gatedstack import Fp8GatedMlpStack
from tests import block_norm_reference as RN
from tests import glu_reference as RG

pytestmark = pytest.mark.gpu

M, D, K = 256, 128, 352
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def make(layers, alphas=True, gated=True, act=B.ACT_SILU):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    params = [((1 + 0.1 * r(D)).cuda(), (0.5 + 0.1 * r(D)).cuda(), torch.tensor([0.95 - 0.1 * i]).cuda() if alphas else None,
               (r(D, 2 * K) / D ** 0.5).bfloat16().cuda(), (r(K, D) / K ** 0.5).bfloat16().cuda()) for i in range(layers)]
    gates = [torch.sigmoid(r(M)).cuda() if gated else None for _ in range(layers)]
    x, dout = r(M, D).bfloat16().cuda(), (1e-2 * r(M, D)).bfloat16().cuda()
    return Fp8GatedMlpStack(M, D, K, layers, act=act), params, gates, x, dout


def rel(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().cpu().norm())


def ones():
    return torch.ones(M, dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("layers,alphas,gated", [(1, False, False), (1, True, True), (3, True, True), (2, True, False)])
def test_step_against_its_parts_and_the_model(layers, alphas, gated):
    s, params, gates, x, dout = make(layers, alphas, gated)
    out = s.forward(x, params, gates, calibrate=True)
    dx, grads = s.backward(dout, params, gates, calibrate=True)
    torch.cuda.synchronize()
    assert s.gemm_status.item() == 0
    assert torch.equal(s.layers[0].r, x)
    bf = torch.bfloat16
    for i, L in enumerate(s.layers):
        weight, post, alpha, W1, W2 = params[i]
        y, rstd, ty, tr = RN.norm(L.r.double(), weight.double(), s.eps)
        RN.assert_within(L.n, y, RN.rounded(y, ty, bf), "n")
        RN.assert_within(L.rstd, rstd, tr, "rstd")
        sn, sa, sw1, sw2 = (d.last_scale for d in L.scales())
        assert torch.equal(L.n_q, RG.codes_of(L.n, sn, E4)[0])
        g, u, a, tg, tu, ta = RG.fwd(L.n_q.view(E4).double() / sn.double(), L.w1_q_t.view(E4).double() / sw1.double(), "silu")
        RG.assert_within(L.h, torch.cat([g, u], 1), torch.cat([tg, tu], 1), "h")
        assert torch.equal(L.a_q_t, L.a_q.t())
        # the product's codes: within a code's half step of the 64-bit product, beside its BF16 tolerance
        RG.assert_within(L.a_q.view(E4).double() / sa.double(), a, ta * 1.1 + a.abs() * 2.0 ** -4 + 2.0 ** -10 / sa.double(), "a_q")
        gate, al = gates[i].double() if gated else ones(), float(alpha) if alphas else 1.0
        want, rp, tr, trp = RN.stream(L.branch.double(), L.r.double(), post.double(), gate, al, True, s.eps)
        RN.assert_within(s.layers[i + 1].r if i + 1 < layers else out, want, RN.rounded(want, tr, bf), "r")
        RN.assert_within(L.rstd_post, rp, trp, "rstd_post")
    dres = dout
    for i in range(layers - 1, -1, -1):
        L = s.layers[i]
        weight, post, alpha, W1, W2 = params[i]
        sn, sa, sw1, sw2 = (d.last_scale for d in L.scales())
        sdb, sdh = L.db_s.last_scale, L.dh_s.last_scale
        dh, tol = RG.bwd(L.db_q.view(E5).double() / sdb.double(), L.w2_q.view(E4).double() / sw2.double(), L.h.double(), "silu")
        RG.assert_within(L.dh_q.view(E5).double() / sdh.double(), dh, tol * 1.2 + dh.abs() * 2.0 ** -3 + 2.0 ** -17 / sdh.double(), "dh_q")
        assert torch.equal(L.dh_q_t, L.dh_q.t())
        # the pass between this block and the sub-layer's end below it
        below = s.layers[i - 1] if i else None
        gate = gates[i - 1].double() if gated and i else ones()
        al = float(params[i - 1][2]) if alphas and i else 1.0
        want = RN.bwd(L.dn.double(), L.r.double(), L.rstd.double(), weight.double(), dres_in(s, i, dout).double(),
                      below.branch.double() if i else L.r.double(), below.rstd_post.double() if i else None,
                      params[i - 1][1].double() if i else torch.ones(D, dtype=torch.float64, device="cuda"), gate, al,
                      below.r.double() if i and alphas else None, bool(i))
        v, t = want["dresidual"]
        RN.assert_within(L.dr, v, RN.rounded(v, t, bf), "dr")
        RN.assert_within(grads[i][0], *want["dweight"], "dweight")
        if i:
            v, t = want["dx"]
            RN.assert_within(below.db, v, RN.rounded(v, t, bf), "branch gradient below")
            RN.assert_within(grads[i - 1][1], *want["dpost_weight"], "dpost_weight")
            if alphas:
                RN.assert_within(grads[i - 1][2], *want["dalpha"], "dalpha")
            if gated:
                RN.assert_within(grads[i - 1][5], *want["dgate"], "dgate")
    assert torch.equal(dx, s.layers[0].dr)

    # the model in float64
    names = [(i, j) for i in range(layers) for j in range(5) if params[i][j] is not None]
    leaf = {k: params[k[0]][k[1]].double().cpu().requires_grad_() for k in names}
    gl = [gates[i].double().cpu().requires_grad_() if gated else torch.ones(M, dtype=torch.float64) for i in range(layers)]
    x64 = x.double().cpu().requires_grad_()
    y = x64
    rms = lambda v: v * (v.square().mean(1, keepdim=True) + s.eps).rsqrt()  # noqa: E731
    for i in range(layers):
        h = rms(y) * leaf[i, 0] @ leaf[i, 3]
        b = (torch.nn.functional.silu(h[:, :K]) * h[:, K:]) @ leaf[i, 4]
        y = leaf.get((i, 2), 1.0) * y + gl[i][:, None] * (rms(b) * leaf[i, 1])
    y.backward(dout.double().cpu())
    assert rel(out, y.detach()) < 0.12
    assert rel(dx, x64.grad) < 0.25
    for i, j in names:
        assert rel(grads[i][j], leaf[i, j].grad) < 0.25, (i, j)
    for i in range(layers if gated else 0):
        assert rel(grads[i][5], gl[i].grad) < 0.25, i


def dres_in(s, i, dout):
    """The stream's gradient that reaches sub-layer i from above its norm."""
    return s.dr if i + 1 == len(s.layers) else s.layers[i + 1].dr


def flat(out, dx, grads):
    return [out.clone(), dx.clone()] + [t.clone() for g in grads for t in g if t is not None]


@pytest.mark.parametrize("steps", [1, 2, 3])
def test_captured_steps_carry_the_scales(steps):
    """A graph of any number of steps does what eager steps do, also with eager steps between its replays."""
    s, params, gates, x, dout = make(2)
    t = make(2)[0]

    def step(k, x, dout, **kw):
        out = k.forward(x, params, gates, **kw)
        return (out, *k.backward(dout, params, gates, **kw))

    x_in, d_in = x.clone(), dout.clone()
    step(s, x, dout, calibrate=True), step(t, x_in, d_in, calibrate=True)
    step(s, x, dout), step(t, x_in, d_in)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(steps):
            captured = step(t, x_in, d_in)
    for turn in range(5):
        xk, dk = x * 1.5 ** (turn + 1), dout * 0.5 ** (turn + 1)
        x_in.copy_(xk)
        d_in.copy_(dk)
        if turn == 3:
            got, want = step(t, x_in, d_in), step(s, xk, dk)
        else:
            g.replay()
            got = captured
            for _ in range(steps):
                want = step(s, xk, dk)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(*got), flat(*want), strict=True)), turn


@pytest.mark.parametrize("act", [B.ACT_GELU, B.ACT_RELU2, B.ACT_RELU, B.ACT_IDENTITY])
def test_activations_run_and_have_gradients(act):
    s, params, gates, x, dout = make(1, act=act)
    out = s.forward(x, params, gates, calibrate=True)
    dx, grads = s.backward(dout, params, gates, calibrate=True)
    assert s.gemm_status.item() == 0
    assert all(bool(torch.isfinite(t).all()) and bool(t.any()) for t in [out, dx, *grads[0]])


def test_backward_does_not_need_the_callers_x():
    s, params, gates, x, dout = make(2)
    t = make(2)[0]
    want = flat(s.forward(x, params, gates, calibrate=True).clone(), *s.backward(dout, params, gates, calibrate=True))
    mine = x.clone()
    out = t.forward(mine, params, gates, calibrate=True).clone()
    mine.fill_(float("nan"))
    assert all(torch.equal(a, b) for a, b in zip(flat(out, *t.backward(dout, params, gates, calibrate=True)), want, strict=True))
    again = s.forward(want[0], params, gates).clone()
    assert torch.equal(t.forward(t.out, params, gates), again)
