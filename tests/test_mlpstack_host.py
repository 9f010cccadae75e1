"""Fp8MlpStack's checks of its arguments, which need no GPU: nothing is launched."""
import pytest
import torch

from quantize_fp8_gemm_gb300.mlpstack import Fp8MlpStack

M, D, K = 32, 16, 48


@pytest.fixture(scope="module")
def stack():
    from quantize_fp8_gemm_gb300 import build
    build.build()
    return Fp8MlpStack(M, D, K, 2, device="cpu")


def layer(**kw):
    p = dict(weight=torch.ones(D), bias=torch.zeros(D), w1=torch.zeros(D, K, dtype=torch.bfloat16),
             w2=torch.zeros(K, D, dtype=torch.bfloat16))
    return tuple({**p, **kw}.values())


X = torch.zeros(M, D, dtype=torch.bfloat16)


@pytest.mark.parametrize("count", [0, 1, 3])
def test_one_tuple_of_parameters_a_sub_layer(stack, count):
    """Neither a shorter stack than was built nor parameters left over."""
    with pytest.raises(ValueError, match="2 sub-layers"):
        stack.forward(X, [layer() for _ in range(count)])
    with pytest.raises(ValueError, match="2 sub-layers"):
        stack.backward(X, [layer() for _ in range(count)])


def matrix(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("bad,kind,what", [
    (dict(w1=matrix(K, D)), ValueError, "W1"),  # transposed: the same bytes
    (dict(w2=matrix(D, K)), ValueError, "W2"),
    (dict(w1=matrix(D, K // 2)), ValueError, "W1"),  # fits the buffers, and fills a part of them
    (dict(w2=matrix(K, D, dtype=torch.float32)), TypeError, "W2 must be torch.bfloat16"),
    (dict(w1=matrix(D, K, dtype=torch.float16)), TypeError, "W1 must be torch.bfloat16"),
])
def test_matrices_of_the_stacks_shape_and_type(stack, bad, kind, what):
    with pytest.raises(kind, match=what):
        stack.forward(X, [layer(), layer(**bad)])
    with pytest.raises(kind, match=what):
        stack.backward(X, [layer(**bad), layer()])
