"""Layer norm and dropout among the FP8 GEMMs as a training step uses them (Fp8MlpStack).

Each pass between two GEMMs is checked against the 64-bit reference from the tensors that
the step itself fed it; the stack as a whole against the float64 model of the same weights.
The second check's bound: an operand in E4M3 is off by 2.7 % RMS (the pages' own experiment,
tests/golden/outlier_experiment.txt), in E5M2 by twice that, independently per element, so a
product of two E4M3 operands by 3.8 %, and of an E4M3 and an E5M2 one by 6 %.  The branch has
two such products and the squared ReLU between them doubles the first one's share:
sqrt((2 * 3.8)^2 + 3.8^2) = 8.5 %.  A gradient passes two products more, and the activation's
derivative with the error of H: sqrt(8.5^2 + 3.8^2 + 6^2 + 6^2) = 12.6 %; one sub-layer above
adds its own.  0.12 and 0.25 leave room for the sampling of the errors."""
import numpy as np
import pytest
import torch

from quantize_fp8_gemm_gb300 import binding as B
from quantize_fp8_gemm_gb300.mlpstack import Fp8MlpStack
from tests import norm_reference as R
from tests.norm_reference import assert_within, f64

pytestmark = pytest.mark.gpu

M, D, K, P, SEED = 256, 128, 512, 0.1, 77


def make(layers):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    params = [((1 + 0.1 * r(D)).cuda(), (0.1 * r(D)).cuda(), (r(D, K) / D ** 0.5).bfloat16().cuda(),
               (r(K, D) * 0.7 / K ** 0.5).bfloat16().cuda()) for _ in range(layers)]
    x, dout = r(M, D).bfloat16().cuda(), (1e-2 * r(M, D)).bfloat16().cuda()
    return Fp8MlpStack(M, D, K, layers, p=P, seed=SEED), params, x, dout


def masks(layers, step=0):
    return [R.keep_mask(SEED, i + (step << 32), M, D, P) for i in range(layers)]


def rel(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().cpu().norm())


@pytest.mark.parametrize("layers", [1, 3])
def test_step_against_its_parts_and_the_model(layers):
    s, params, x, dout = make(layers)
    out = s.forward(x, params, calibrate=True)
    dx, grads = s.backward(dout, params, calibrate=True)
    torch.cuda.synchronize()
    assert s.gemm_status.item() == 0
    keep = masks(layers)
    r = x.cpu()
    for i, L in enumerate(s.layers):  # forward: the residual stream exactly, the norm within its tolerance
        assert torch.equal(L.r.cpu(), r)
        w, b = f64(params[i][0]), f64(params[i][1])
        want, tol = R.norm_fwd(f64(L.r), w, b, 1e-5), R.fwd_tolerances(f64(L.r), w, b, 1e-5, torch.bfloat16)
        for got, v, t, name in zip((L.n, L.mean, L.rstd), want, tol, ("n", "mean", "rstd")):
            assert_within(f64(got), v, t, name)
        q = torch.empty_like(L.n_q)
        B.fp8_quant_fused(L.n, B.ACT_IDENTITY, B.E4M3, L.n_s.last_scale, q_out=q)
        assert torch.equal(q, L.n_q)
        r = R.residual_stream(L.branch.cpu(), r, keep[i], P)
    assert torch.equal(out.cpu(), r)
    inv = 1.0 / (1.0 - P)
    dres = dout
    assert torch.equal(s.layers[-1].db.cpu(), R.residual_stream(dout.cpu(), None, keep[-1], P))
    for i in range(layers - 1, -1, -1):  # backward
        L = s.layers[i]
        args = (f64(L.dn), f64(L.r), f64(L.mean), f64(L.rstd), f64(params[i][0]), f64(dres))
        dr, dw, db = R.norm_bwd(*args)
        t_dx, t_db, t_dw, t_dbias = R.bwd_tolerances(*args, torch.bfloat16, inv)
        assert_within(f64(L.dr), dr, t_dx, "dr")
        assert_within(f64(grads[i][0]), dw, t_dw, "dweight")
        assert_within(f64(grads[i][1]), db, t_dbias, "dbias")
        if i:
            assert_within(f64(s.layers[i - 1].db), np.where(keep[i - 1], dr * inv, 0.0), t_db, "branch gradient below")
        dres = L.dr
    assert torch.equal(dx, s.layers[0].dr)

    # the model in float64
    leaves = [t.double().cpu().requires_grad_() for p in params for t in p]
    x64 = x.double().cpu().requires_grad_()
    y = x64
    for i in range(layers):
        w, b, w1, w2 = leaves[4 * i:4 * i + 4]
        n = torch.nn.functional.layer_norm(y, (D,), w, b, 1e-5)
        y = y + (torch.relu(n @ w1).square() @ w2) * torch.from_numpy(keep[i]) * inv
    y.backward(dout.double().cpu())
    assert rel(out, y.detach()) < 0.12
    assert rel(dx, x64.grad) < 0.25
    for i in range(layers):
        for j, name in enumerate(("dweight", "dbias", "dW1", "dW2")):
            assert rel(grads[i][j], leaves[4 * i + j].grad) < 0.25, (i, name)


def test_steps_take_new_masks_and_a_graph_replays_them():
    """Two eager steps warm the delayed scales; then a captured step with advance() in it: each
    replay has the masks of its own step."""
    s, params, x, dout = make(2)
    s.forward(x, params, calibrate=True)
    s.backward(dout, params, calibrate=True)
    s.advance()
    first = s.forward(x, params).clone()
    keep = masks(2, step=1)
    assert torch.equal(first.cpu(), R.residual_stream(s.layers[1].branch.cpu(), s.layers[1].r.cpu(), keep[1], P))
    s.backward(dout, params)
    s.advance()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # two steps: the scale slots alternate
        for _ in range(2):
            out = s.forward(x, params)
            s.backward(dout, params)
            s.advance()
    for replay in range(2):
        g.replay()
        torch.cuda.synchronize()
        step = 3 + 2 * replay  # the second of the replay's steps is the one still in the buffers
        L = s.layers[1]
        assert torch.equal(out.cpu(), R.residual_stream(L.branch.cpu(), L.r.cpu(), masks(2, step)[1], P))
        assert s.gemm_status.item() == 0 and all(int(d.status.item()) == 0 for l in s.layers for d in l.scales())


def test_refusals():
    for bad in (dict(M=100), dict(D=100), dict(K=100), dict(layers=0)):
        with pytest.raises(ValueError):
            Fp8MlpStack(**{**dict(M=64, D=64, K=64, layers=1), **bad})
