"""What Fp8MlpStack keeps between its calls."""
import pytest
import torch

from tests.test_mlpstack_gpu import make

pytestmark = pytest.mark.gpu


def flat(dx, grads):
    return [dx.clone()] + [t.clone() for g in grads for t in g]


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
