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
