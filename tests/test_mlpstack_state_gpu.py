"""What Fp8MlpStack keeps between its calls: the caller's x, and the delayed scales under CUDA graphs."""
import pytest
import torch

from tests.test_mlpstack_gpu import make

pytestmark = pytest.mark.gpu


def flat(dx, grads):
    return [dx.clone()] + [t.clone() for g in grads for t in g]


def scales_of(s):
    return [t.clone() for L in s.layers for d in (*L.scales(), L.db_s, L.dh_s) for t in (d.scale, d.history, d.status)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("layers", [1, 2])
def test_backward_does_not_need_the_callers_x(layers):
    """x may change between forward and backward, and may be the stack's own output."""
    s, params, x, dout = make(layers)
    t = make(layers)[0]
    want = s.forward(x, params, calibrate=True).clone()
    want_grads = flat(*s.backward(dout, params, calibrate=True))
    mine = x.clone()
    assert torch.equal(t.forward(mine, params, calibrate=True), want)
    mine.fill_(float("nan"))
    assert same(flat(*t.backward(dout, params, calibrate=True)), want_grads)
    # a second application to the first one's output, which is the buffer that it writes
    kept = want.clone()
    want2 = s.forward(kept, params).clone()
    want_grads2 = flat(*s.backward(dout, params))
    assert torch.equal(t.forward(t.out, params), want2)
    assert same(flat(*t.backward(dout, params)), want_grads2)


def step(s, x, params, dout):
    out = s.forward(x, params)
    dx, grads = s.backward(dout, params)
    s.advance()
    return out, dx, grads


@pytest.mark.parametrize("steps", [1, 2, 3])
def test_captured_steps_carry_the_scales(steps):
    """A graph of any number of steps does what eager steps do, also with eager steps between its
    replays: x grows from step to step, so that a scale that stood still would show."""
    s, params, x, dout = make(2)
    t = make(2)[0]
    for k in (s, t):
        k.forward(x, params, calibrate=True)
        k.backward(dout, params, calibrate=True)
        k.advance()
    x_in, d_in = x.clone(), dout.clone()
    step(t, x_in, params, d_in)
    step(s, x, params, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(steps):
            captured = step(t, x_in, params, d_in)
    for turn in range(6):
        xk, dk = x * 1.5 ** (turn + 1), dout * 0.5 ** (turn + 1)
        x_in.copy_(xk)
        d_in.copy_(dk)
        if turn == 3:
            got = step(t, x_in, params, d_in)
            want = step(s, xk, params, dk)
        else:
            g.replay()
            got = captured
            for _ in range(steps):
                want = step(s, xk, params, dk)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]), turn
        assert same(flat(*got[1:]), flat(*want[1:])), turn
        assert same(scales_of(t), scales_of(s)), turn


def test_a_scale_seeded_by_hand_between_replays():
    s, params, x, dout = make(1)
    t = make(1)[0]
    for k in (s, t):
        k.forward(x, params, calibrate=True)
        k.backward(dout, params, calibrate=True)
        k.advance()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(t, x, params, dout)
    for amax in (40.0, 3.0):
        for k in (s, t):
            k.layers[0].n_s.seed(amax)
        assert t.layers[0].n_s.scale.item() == torch.tensor(448.0 / (2.0 * amax)).item()  # in float32
        g.replay()
        want = step(s, x, params, dout)
        torch.cuda.synchronize()
        assert torch.equal(captured[0], want[0]) and same(flat(*captured[1:]), flat(*want[1:]))
        assert same(scales_of(t), scales_of(s))
