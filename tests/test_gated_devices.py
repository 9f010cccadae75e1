"""The gated block's and the block norms' calls run on the current device: a tensor of another one is refused by
name, whichever argument it is, before anything is launched.  No GPU: the tensors are stand-ins without memory."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from quantize_fp8_gemm_gb300 import binding as B

M, N, F, K = 16, 32, 48, 64
BF, F32, U8, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64
ROWS, COLS, TOKENS, CELL, COUNT = ((M, N), BF), ((N,), F32), ((M,), F32), ((1,), F32), ((1,), I64)
STATUS = ((1,), torch.int32)
CALLS = {
    "block_norm_fwd": dict(x=ROWS, weight=COLS, y=ROWS, rstd=TOKENS, residual=ROWS, alpha=CELL, gate=TOKENS, post_weight=COLS,
                           rstd_post=TOKENS, r_out=ROWS, scale=CELL, q_out=((M, N), U8), amax_out=CELL, sat_count=COUNT),
    "block_norm_bwd": dict(dy=ROWS, r=ROWS, rstd=TOKENS, weight=COLS, dr=ROWS, x=ROWS, residual=ROWS, alpha=CELL, gate=TOKENS,
                           post_weight=COLS, rstd_post=TOKENS, dresidual=ROWS, dx=ROWS, dweight=COLS, dpost_weight=COLS, dgate=TOKENS,
                           dalpha=CELL, workspace=((4096,), U8)),
    "fp8_glu_fwd": dict(x_q=((M, K), U8), w1t_q=((2 * F, K), U8), scale_x=CELL, scale_w=CELL, h_out=((M, 2 * F), BF), act_out=((M, F), BF),
                        scale_a=CELL, a_q=((M, F), U8), a_q_t=((F, M), U8), amax_out=CELL, sat_count=COUNT, status=STATUS),
    "fp8_gemm_dgrad_glu": dict(dy_q=((M, N), U8), w2_q=((F, N), U8), scale_dy=CELL, scale_w=CELL, h=((M, 2 * F), BF), dh=((M, 2 * F), BF),
                               scale_dh=CELL, dh_q=((M, 2 * F), U8), dh_q_t=((2 * F, M), U8), amax_out=CELL, sat_count=COUNT, status=STATUS),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, args in CALLS.items() for n in args])
def test_a_tensor_of_another_device_is_refused(monkeypatch, call, name):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # a stand-in's address is asked for
        args = {n: torch.empty(shape, dtype=dtype, device=f"cuda:{int(n == name)}") for n, (shape, dtype) in CALLS[call].items()}
        with pytest.raises(ValueError, match=rf"^{name} is on cuda:1, the current device is cuda:0$"):
            getattr(B, call)(**args, stream=object())
