"""A stack of GPT-2-style MLP sub-layers in FP8, forward and backward:

    x_{l+1} = x_l + dropout( act( layer_norm(x_l) . W1_l ) . W2_l )

Every product runs on the FP8 GEMMs with delayed per-tensor scales ("FP8 Training
& Inference", FP8 Training Recipe: weights and activations in E4M3, gradients in
E5M2), and what stands between them is one pass over the data each:

    layer_norm_fwd   the previous sub-layer's dropout and residual addition, the norm, and
                     the E4M3 codes that the up-projection reads
    fp8_upproj_fwd   H = codes . W1, and act(H) quantized in its epilogue
    fp8_gemm_fwd     the branch act(H) . W2
    dropout_fwd      dropout and residual of the last sub-layer (no norm follows it)

and back again: dropout_bwd, the gradient's casts, fp8_gemm_dgrad_act, the weight
gradients, fp8_gemm_dgrad, and layer_norm_bwd, which adds the residual's gradient
and forms the branch gradient of the sub-layer below.  No dropout mask is stored:
each sub-layer has its own offset of the generator, and a backward pass forms the
forward's masks again; ``advance()`` gives the next step new ones.  Nothing of a step's
state is on the host: a CUDA graph may hold any number of steps, and its replays may
mix with eager ones.

Like ``Fp8DownProj`` this module owns buffers and the order of the calls; the
arithmetic is libfp8q's.
"""
from __future__ import annotations

import torch

from . import binding as B
from .downproj import DelayedScale


class _Scale(DelayedScale):
    """A DelayedScale whose state between two steps is always in slot 1.

    DelayedScale alternates its slots by a switch on the host, which a CUDA graph would freeze.
    Here begin() moves the state to slot 0, a step casts with slot 0, and update() writes slot 1:
    so a captured step starts where the step before it, eager or replayed, ended."""

    def __init__(self, fmt: int, margin: float, history_len: int, device, record: torch.Tensor):
        super().__init__(fmt, margin, history_len, device)
        self.record = record  # int64 [slot][(scale, amax), count]
        words = record.view(torch.float32)
        self.scales, self.amaxes, self.sats = words[:, 0], words[:, 1], record[:, 1]
        self.scales.fill_(1.0)
        self.slot = 1

    def begun(self) -> None:
        self.slot, self.clean = 0, True

    def begin(self) -> None:
        self.record[0].copy_(self.record[1])
        self.begun()

    def seed(self, amax: float) -> None:
        self.begin()
        super().seed(amax)


class _Scales:
    """The scales that one pass over the stack casts with, begun by one copy."""

    def __init__(self, fmt: int, count: int, margin: float, history_len: int, device):
        self.records = torch.zeros(count, 2, 2, dtype=torch.int64, device=device)
        self.scales = [_Scale(fmt, margin, history_len, device, r) for r in self.records]

    def begin(self) -> None:
        self.records[:, 0].copy_(self.records[:, 1])
        for s in self.scales:
            s.begun()


class _Layer:
    """Buffers of one sub-layer of M tokens, width D, hidden width K, and its scales: of the norm's output, the
    activation, W1 and W2 in the forward pass, of the branch's and the activation's gradient in the backward."""

    def __init__(self, M: int, D: int, K: int, forward_scales, backward_scales, seed: int, index: int, device):
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
        q8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=device)  # noqa: E731
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=device)  # noqa: E731
        self.n_s, self.h_s, self.w1_s, self.w2_s = forward_scales
        self.db_s, self.dh_s = backward_scales
        # (seed, offset): sub-layers of one step differ in the offset's low half, steps in its high half
        self.rng = torch.tensor([seed, index], dtype=torch.int64, device=device)
        # forward
        self.r, self.n, self.n_q = bf(M, D), bf(M, D), q8(M, D)
        self.mean, self.rstd = f32(M), f32(M)
        self.h, self.a, self.a_q = bf(M, K), bf(M, K), q8(M, K)
        self.w1_q, self.w1_q_t = q8(D, K), q8(K, D)
        self.w2_q, self.w2_q_t = q8(K, D), q8(D, K)
        self.branch = bf(M, D)
        # backward
        self.db, self.db_q, self.db_q_t = bf(M, D), q8(M, D), q8(D, M)
        self.dh, self.dh_q, self.dh_q_t = bf(M, K), q8(M, K), q8(K, M)
        self.n_q_t, self.a_q_t = q8(D, M), q8(K, M)
        self.dn, self.dr = bf(M, D), bf(M, D)
        self.dw1, self.dw2 = bf(D, K), bf(K, D)
        self.dweight, self.dbias = f32(D), f32(D)

    def scales(self):
        return (self.n_s, self.h_s, self.w1_s, self.w2_s)


class Fp8MlpStack:
    """``layers`` sub-layers on [M, D] BF16 activations with hidden width K.

    Parameters of sub-layer l, passed to the calls as ``params[l]``: a tuple
    (weight [D], bias [D], W1 [D,K] BF16, W2 [K,D] BF16), the layer norm's in
    float32 or BF16.  M, D and K are multiples of 16 (the FP8 GEMMs' rule)."""

    def __init__(self, M: int, D: int, K: int, layers: int = 1, *, p: float = 0.1, eps: float = 1e-5,
                 act: int = B.ACT_RELU2, margin: float = 2.0, history_len: int = 1, seed: int = 0, device="cuda"):
        if layers < 1 or M % 16 or D % 16 or K % 16:
            raise ValueError("layers >= 1, and M, D, K multiples of 16")
        self.M, self.D, self.K, self.p, self.eps, self.act = M, D, K, float(p), float(eps), act
        self.forward_scales = _Scales(B.E4M3, 4 * layers, margin, history_len, device)
        self.backward_scales = _Scales(B.E5M2, 2 * layers, margin, history_len, device)
        self.layers = [_Layer(M, D, K, self.forward_scales.scales[4 * i:4 * i + 4],
                              self.backward_scales.scales[2 * i:2 * i + 2], seed, i, device) for i in range(layers)]
        self.out = torch.empty(M, D, dtype=torch.bfloat16, device=device)
        self.workspace = torch.empty(B.layer_norm_bwd_workspace_bytes(M, D), dtype=torch.uint8, device=device)
        self.gemm_status = torch.zeros(1, dtype=torch.int32, device=device)

    def _checked(self, params) -> list:
        """The sub-layers' parameters, one tuple each.  (The quantize takes a matrix as raw BF16 of any
        shape that fits its outputs, and the layer norm checks its own vectors.)"""
        params = list(params)
        if len(params) != len(self.layers):
            raise ValueError(f"{len(params)} tuples of parameters for {len(self.layers)} sub-layers")
        for _, _, W1, W2 in params:
            for W, shape, name in ((W1, (self.D, self.K), "W1"), (W2, (self.K, self.D), "W2")):
                if W.dtype != torch.bfloat16:
                    raise TypeError(f"{name} must be torch.bfloat16, not {W.dtype}")
                if W.shape != shape:
                    raise ValueError(f"{name} is {list(W.shape)}, the stack needs {list(shape)}")
        return params

    def _cast(self, s: DelayedScale, cast, calibrate: bool) -> None:
        """cast(scale, amax, sat, flags); with calibrate first once for its amax alone, which seeds the scale."""
        for _ in range(2 if calibrate else 1):
            cast(s.scale, s.amax, s.sat, B.ACCUMULATE if s.clean else 0)
            s.clean = False
            if calibrate:
                calibrate = False
                s.update()
                s.begin()

    def forward(self, x: torch.Tensor, params, *, calibrate: bool = False) -> torch.Tensor:
        """The stack's output [M, D], a buffer of the stack that the next forward() writes; x may be that
        buffer, and may change as soon as the call's work on the stream is done.  ``calibrate``: take each
        tensor's scale from its own values (a first step, whose histories are empty)."""
        params = self._checked(params)
        self.forward_scales.begin()
        before = None
        for L, (weight, bias, W1, W2) in zip(self.layers, params):
            for W, s, q, q_t in ((W1, L.w1_s, L.w1_q, L.w1_q_t), (W2, L.w2_s, L.w2_q, L.w2_q_t)):
                self._cast(s, lambda sc, am, sat, fl: B.fp8_quant_fused_ex(
                    W, B.ACT_IDENTITY, B.E4M3, sc, q_out=q, q_t_out=q_t, amax_out=am, sat_count=sat, flags=fl), calibrate)
            if before is None:  # r = x, kept for backward in the same pass: the caller may change x
                into = dict(x=x, r_out=L.r)
            else:  # the dropout and residual of the sub-layer below, in the same pass
                into = dict(x=before.branch, residual=before.r, r_out=L.r, p=self.p, rng=before.rng)
            self._cast(L.n_s, lambda sc, am, sat, fl: B.layer_norm_fwd(
                weight=weight, bias=bias, y=L.n, eps=self.eps, mean=L.mean, rstd=L.rstd, fmt=B.E4M3, scale=sc,
                q_out=L.n_q, amax_out=am, sat_count=sat, flags=fl, **into), calibrate)
            self._cast(L.h_s, lambda sc, am, sat, fl: B.fp8_upproj_fwd(
                L.n_q, L.w1_q_t, L.n_s.scale, L.w1_s.scale, sc, L.a_q, act=self.act, h_out=L.h, act_out=L.a,
                amax_out=am, sat_count=sat, flags=fl, status=self.gemm_status), calibrate)
            B.fp8_gemm_fwd(L.a_q, L.w2_q_t, L.h_s.scale, L.w2_s.scale, L.branch, status=self.gemm_status)
            for s in L.scales():
                s.update()
            before = L
        B.dropout_fwd(before.branch, self.out, self.p, before.rng, residual=before.r)
        return self.out

    def backward(self, dout: torch.Tensor, params, *, calibrate: bool = False):
        """(dx, grads) of the last forward(): dx [M, D], and per sub-layer (dweight, dbias, dW1, dW2); buffers
        of the stack, which the next backward() writes."""
        params = self._checked(params)
        self.backward_scales.begin()
        last = self.layers[-1]
        B.dropout_bwd(dout, last.db, self.p, last.rng)
        dres, grads = dout, []
        for i in range(len(self.layers) - 1, -1, -1):
            L, below = self.layers[i], self.layers[i - 1] if i else None
            weight = params[i][0]
            sn, sh, sw1, sw2 = (s.last_scale for s in L.scales())
            self._cast(L.db_s, lambda sc, am, sat, fl: B.fp8_quant_fused_ex(
                L.db, B.ACT_IDENTITY, B.E5M2, sc, q_out=L.db_q, q_t_out=L.db_q_t, amax_out=am, sat_count=sat,
                flags=fl), calibrate)
            B.fp8_gemm_dgrad_act(L.db_q, L.w2_q, L.db_s.scale, sw2, L.h, L.dh, act=self.act, status=self.gemm_status)
            B.fp8_quant_fused(L.a, B.ACT_IDENTITY, B.E4M3, sh, q_t_out=L.a_q_t)
            B.fp8_gemm_wgrad(L.a_q_t, L.db_q_t, sh, L.db_s.scale, L.dw2, status=self.gemm_status)
            self._cast(L.dh_s, lambda sc, am, sat, fl: B.fp8_quant_fused_ex(
                L.dh, B.ACT_IDENTITY, B.E5M2, sc, q_out=L.dh_q, q_t_out=L.dh_q_t, amax_out=am, sat_count=sat,
                flags=fl), calibrate)
            B.fp8_gemm_dgrad(L.dh_q, L.w1_q, L.dh_s.scale, sw1, L.dn, status=self.gemm_status)
            B.fp8_quant_fused(L.n, B.ACT_IDENTITY, B.E4M3, sn, q_t_out=L.n_q_t)
            B.fp8_gemm_wgrad(L.n_q_t, L.dh_q_t, sn, L.dh_s.scale, L.dw1, status=self.gemm_status)
            # the norm's gradient, the residual's added; and the branch gradient of the sub-layer below
            drop = {} if below is None else dict(p=self.p, rng=below.rng, dbranch=below.db)
            B.layer_norm_bwd(L.dn, L.r, L.mean, L.rstd, weight, L.dr, dresidual=dres, dweight=L.dweight, dbias=L.dbias,
                             workspace=self.workspace, **drop)
            L.db_s.update()
            L.dh_s.update()
            dres = L.dr
            grads.append((L.dweight, L.dbias, L.dw1, L.dw2))
        return dres, grads[::-1]

    def advance(self) -> None:
        """New dropout masks for the next step (on the device: a captured step may contain it)."""
        for L in self.layers:
            L.rng[1:] += 1 << 32
