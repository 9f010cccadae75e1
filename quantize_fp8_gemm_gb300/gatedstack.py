"""A stack of gated MLP sub-layers in FP8 with norms before and after each block, forward and backward:

    r_{l+1} = alpha_l r_l + gate_l norm( (act(n Wg_l) * (n Wu_l)) W2_l ) wp_l,   n = norm(r_l) w_l

Norms are root-mean-square ones; W1 = [Wg | Wu] is one matrix, so its gradient and its input's are
those of a linear layer.  Products run on the FP8 GEMMs with delayed per-tensor scales as in
``Fp8MlpStack``; in the forward pass the data is passed over once between two of them:

    block_norm_fwd      the sub-layer's end below (norm, gate, residual), the norm before this
                        block, and the E4M3 codes that the projections read
    fp8_glu_fwd         both projections, the activation, the product and its codes, in the
                        layouts of the down-projection and of its weight gradient
    fp8_gemm_fwd        the branch

and back: block_norm_bwd, the branch gradient's cast, fp8_gemm_dgrad_glu (whose epilogue writes the
projections' gradients as E5M2 codes in both layouts: they never exist in BF16), the weight
gradients, fp8_gemm_dgrad, block_norm_bwd.  Two passes there stand by themselves: the cast of the branch
gradient, which block_norm_bwd writes in BF16, and that of the norm's output into the transposed codes that
W1's gradient reads, for which the forward keeps it in BF16.  Nothing of a step's state is on the host: a
CUDA graph may hold any number of steps, and its replays may mix with eager ones.
"""
from __future__ import annotations

import torch

from . import binding as B
from .mlpstack import _Scales


class _Layer:
    """Buffers of one sub-layer of M tokens, width D, hidden width K, and its scales: of the norm's output, the
    product, W1 and W2 in the forward pass, of the branch's and the projections' gradient in the backward."""

    def __init__(self, M: int, D: int, K: int, forward_scales, backward_scales, device):
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
        q8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=device)  # noqa: E731
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=device)  # noqa: E731
        self.n_s, self.a_s, self.w1_s, self.w2_s = forward_scales
        self.db_s, self.dh_s = backward_scales
        # forward
        self.r, self.n, self.n_q = bf(M, D), bf(M, D), q8(M, D)
        self.rstd, self.rstd_post = f32(M), f32(M)
        self.h, self.a_q, self.a_q_t = bf(M, 2 * K), q8(M, K), q8(K, M)
        self.w1_q, self.w1_q_t = q8(D, 2 * K), q8(2 * K, D)
        self.w2_q, self.w2_q_t = q8(K, D), q8(D, K)
        self.branch = bf(M, D)
        # backward
        self.db, self.db_q, self.db_q_t = bf(M, D), q8(M, D), q8(D, M)
        self.dh_q, self.dh_q_t, self.n_q_t = q8(M, 2 * K), q8(2 * K, M), q8(D, M)
        self.dn, self.dr = bf(M, D), bf(M, D)
        self.dw1, self.dw2 = bf(D, 2 * K), bf(K, D)
        self.dweight, self.dpost, self.dalpha, self.dgate = f32(D), f32(D), f32(1), f32(M)

    def scales(self):
        return (self.n_s, self.a_s, self.w1_s, self.w2_s)


class Fp8GatedMlpStack:
    """``layers`` gated sub-layers on [M, D] BF16 activations with hidden width K.

    Parameters of sub-layer l, passed to the calls as ``params[l]``: a tuple (weight [D] of the norm
    before the block, post_weight [D] of the one after it, alpha [1] float32 or None for 1, W1 [D,2K]
    BF16, the gate's K columns first, W2 [K,D] BF16), the norms' in float32 or BF16, of one type.
    ``gates``: None, or per sub-layer None or a gate [M] float32.  M, D and K are multiples of 16 (the
    FP8 GEMMs' rule)."""

    def __init__(self, M: int, D: int, K: int, layers: int = 1, *, eps: float = 1e-5, act: int = B.ACT_SILU,
                 margin: float = 2.0, history_len: int = 1, device="cuda"):
        if layers < 1 or M % 16 or D % 16 or K % 16:
            raise ValueError("layers >= 1, and M, D, K multiples of 16")
        self.M, self.D, self.K, self.eps, self.act = M, D, K, float(eps), act
        self.forward_scales = _Scales(B.E4M3, 4 * layers, margin, history_len, device)
        self.backward_scales = _Scales(B.E5M2, 2 * layers, margin, history_len, device)
        self.layers = [_Layer(M, D, K, self.forward_scales.scales[4 * i:4 * i + 4],
                              self.backward_scales.scales[2 * i:2 * i + 2], device) for i in range(layers)]
        self.out, self.dr = (torch.empty(M, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.workspace = torch.empty(B.block_norm_bwd_workspace_bytes(M, D), dtype=torch.uint8, device=device)
        self.gemm_status = torch.zeros(1, dtype=torch.int32, device=device)

    def _checked(self, params, gates) -> list:
        """(layer, weight, post_weight, alpha, W1, W2, gate) of each sub-layer.  (The quantize takes a matrix as
        raw BF16 of any shape that fits its outputs, and the norms check their own vectors.)"""
        params = list(params)
        gates = [None] * len(self.layers) if gates is None else list(gates)
        for given, what in ((params, "tuples of parameters"), (gates, "gates")):
            if len(given) != len(self.layers):
                raise ValueError(f"{len(given)} {what} for {len(self.layers)} sub-layers")
        for _, _, _, W1, W2 in params:
            for W, shape, name in ((W1, (self.D, 2 * self.K), "W1"), (W2, (self.K, self.D), "W2")):
                if W.dtype != torch.bfloat16:
                    raise TypeError(f"{name} must be torch.bfloat16, not {W.dtype}")
                if W.shape != shape:
                    raise ValueError(f"{name} is {list(W.shape)}, the stack needs {list(shape)}")
        return [(L, *p, g) for L, p, g in zip(self.layers, params, gates)]

    def _cast(self, s, cast, calibrate: bool) -> None:
        """cast(scale, amax, sat, flags); with calibrate first once for its amax alone, which seeds the scale."""
        for _ in range(2 if calibrate else 1):
            cast(s.scale, s.amax, s.sat, B.ACCUMULATE if s.clean else 0)
            s.clean = False
            if calibrate:
                calibrate = False
                s.update()
                s.begin()

    def forward(self, x: torch.Tensor, params, gates=None, *, calibrate: bool = False) -> torch.Tensor:
        """The stack's output [M, D], a buffer of the stack that the next forward() writes; x may be that
        buffer, and may change as soon as the call's work on the stream is done.  ``calibrate``: take each
        tensor's scale from its own values (a first step, whose histories are empty)."""
        subs = self._checked(params, gates)
        self.forward_scales.begin()
        into = dict(x=x)  # r = x, kept for backward in the same pass: the caller may change x
        for L, weight, post, alpha, W1, W2, gate in subs:
            for W, s, q, q_t in ((W1, L.w1_s, L.w1_q, L.w1_q_t), (W2, L.w2_s, L.w2_q, L.w2_q_t)):
                self._cast(s, lambda sc, am, sat, fl: B.fp8_quant_fused_ex(
                    W, B.ACT_IDENTITY, B.E4M3, sc, q_out=q, q_t_out=q_t, amax_out=am, sat_count=sat, flags=fl), calibrate)
            self._cast(L.n_s, lambda sc, am, sat, fl: B.block_norm_fwd(
                weight=weight, y=L.n, eps=self.eps, rstd=L.rstd, r_out=L.r, fmt=B.E4M3, scale=sc, q_out=L.n_q,
                amax_out=am, sat_count=sat, flags=fl, **into), calibrate)
            self._cast(L.a_s, lambda sc, am, sat, fl: B.fp8_glu_fwd(
                L.n_q, L.w1_q_t, L.n_s.scale, L.w1_s.scale, act=self.act, h_out=L.h, scale_a=sc, a_q=L.a_q,
                a_q_t=L.a_q_t, amax_out=am, sat_count=sat, flags=fl, status=self.gemm_status), calibrate)
            B.fp8_gemm_fwd(L.a_q, L.w2_q_t, L.a_s.scale, L.w2_s.scale, L.branch, status=self.gemm_status)
            for s in L.scales():
                s.update()
            # the sub-layer's end: in the pass of the norm that follows it
            into = dict(x=L.branch, residual=L.r, alpha=alpha, gate=gate, post_weight=post, post_norm=True,
                        rstd_post=L.rstd_post)
        B.block_norm_fwd(weight=None, y=None, eps=self.eps, r_out=self.out, **into)
        return self.out

    def backward(self, dout: torch.Tensor, params, gates=None, *, calibrate: bool = False):
        """(dx, grads) of the last forward(): dx [M, D], and per sub-layer (dweight, dpost_weight, dalpha, dW1, dW2)
        and with a gate its gradient as well (None in the place of what was None); buffers of the stack, which
        the next backward() writes."""
        subs = self._checked(params, gates)
        self.backward_scales.begin()

        def end_of(i):
            """block_norm_bwd's arguments for the end of sub-layer i."""
            L, _, post, alpha, _, _, gate = subs[i]
            return dict(x=L.branch, residual=None if alpha is None else L.r, alpha=alpha, gate=gate, post_weight=post,
                        post_norm=True, rstd_post=L.rstd_post, dx=L.db, dpost_weight=L.dpost,
                        dgate=None if gate is None else L.dgate, dalpha=None if alpha is None else L.dalpha,
                        workspace=self.workspace)

        B.block_norm_bwd(None, None, None, None, dr=dout, dresidual=self.dr, **end_of(len(subs) - 1))
        dres, grads = self.dr, []
        for i in range(len(subs) - 1, -1, -1):
            L, weight, post, alpha, _, _, gate = subs[i]
            sn, sa, sw1, sw2 = (s.last_scale for s in L.scales())
            self._cast(L.db_s, lambda sc, am, sat, fl: B.fp8_quant_fused_ex(
                L.db, B.ACT_IDENTITY, B.E5M2, sc, q_out=L.db_q, q_t_out=L.db_q_t, amax_out=am, sat_count=sat,
                flags=fl), calibrate)
            self._cast(L.dh_s, lambda sc, am, sat, fl: B.fp8_gemm_dgrad_glu(
                L.db_q, L.w2_q, L.db_s.scale, sw2, L.h, act=self.act, scale_dh=sc, dh_q=L.dh_q, dh_q_t=L.dh_q_t,
                amax_out=am, sat_count=sat, flags=fl, status=self.gemm_status), calibrate)
            B.fp8_gemm_wgrad(L.a_q_t, L.db_q_t, sa, L.db_s.scale, L.dw2, status=self.gemm_status)
            B.fp8_gemm_dgrad(L.dh_q, L.w1_q, L.dh_s.scale, sw1, L.dn, status=self.gemm_status)
            B.fp8_quant_fused(L.n, B.ACT_IDENTITY, B.E4M3, sn, q_t_out=L.n_q_t)
            B.fp8_gemm_wgrad(L.n_q_t, L.dh_q_t, sn, L.dh_s.scale, L.dw1, status=self.gemm_status)
            # this block's norm and the end of the sub-layer below, in one pass
            B.block_norm_bwd(L.dn, L.r, L.rstd, weight, dr=dres, dresidual=L.dr, dweight=L.dweight,
                             **(end_of(i - 1) if i else dict(workspace=self.workspace)))
            L.db_s.update()
            L.dh_s.update()
            dres = L.dr
            grads.append((L.dweight if weight is not None else None, L.dpost if post is not None else None,
                          L.dalpha if alpha is not None else None, L.dw1, L.dw2) + ((L.dgate,) if gate is not None else ()))
        return dres, grads[::-1]
