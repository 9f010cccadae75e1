"""Cases of the gated FP8 MLP: the gated feed-forward kernels and the norms before and after such a block.

One sub-layer is  r' = alpha r + gate norm(mlp(norm(r))) with mlp(y) = (act(y Wg) * (y Wu)) W2.  Measured here:

    glu_fwd   both projections of the E4M3 codes, the activation, the product and its E4M3 codes
              (fp8_glu_fwd)
    glu_bwd   the product's gradient from the down-projection's, and through it both projections'
              pre-activation gradients (fp8_gemm_dgrad_glu)
    bn_fwd    norm after a block, its gate, the scaled residual, norm before the next block and
              its codes (block_norm_fwd)
    bn_bwd    their gradient (block_norm_bwd)

``run`` computes plainly, in float32, with elementary torch operations; with ``own`` set it calls the
framework.  FP8 codes are defined as those of the value rounded to the activations' type, as
everywhere in the framework, and the norm before a block is that of the stored stream r.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAX_MKF = 32768 * 1600 * 6400   # M * K * F of the largest gated case
MAX_ELEMS = 131072 * 1600       # elements of the largest norm case
ACTS = ["silu", "silu", "gelu", "gelu", "relu", "relu2", "identity"]


def listed():
    return [
        # GPT-2-XL, one token of a generating program: the codes alone, nothing is kept
        _glu("glu_fwd_token", "glu_fwd", 1, 1600, 6400, outs="q"),
        # odd counts of rows and of 16-column blocks; the activation in BF16 beside its codes
        _glu("glu_fwd_ragged", "glu_fwd", 1003, 1008, 2736, act="gelu", outs="aq"),
        # GPT-2-XL, a training step's forward: pre-activations kept, codes in both layouts
        _glu("glu_fwd_gpt2xl", "glu_fwd", 32768, 1600, 6400, outs="hqt"),
        # GPT-2-small, one batch, hidden width 8/3 of 768: the gradients' codes in both layouts
        _glu("glu_bwd_gpt2s", "glu_bwd", 8192, 768, 2048, outs="qt"),
        # odd counts, the gradients in BF16
        _glu("glu_bwd_ragged", "glu_bwd", 1003, 1008, 2736, act="gelu", outs="h"),
        # GPT-2-XL, a training step's backward
        _glu("glu_bwd_gpt2xl", "glu_bwd", 32768, 1600, 6400, outs="qt"),
        # GPT-2-XL, one token between two blocks
        _norm("bn_fwd_token", "bn_fwd", 1, 1600, fp8=True),
        # odd width, half precision, rows cut out of a wider buffer, gates by token
        _norm("bn_fwd_ragged", "bn_fwd", 5003, 1001, dtype="fp16", params="fp16", pad=6, gate=True),
        # GPT-2-XL, one large batch between two blocks
        _norm("bn_fwd_gpt2xl", "bn_fwd", 131072, 1600, fp8=True, alpha=True),
        # GPT-2-small, one batch, the residual's scale learned too
        _norm("bn_bwd_gpt2s", "bn_bwd", 8192, 768, alpha=True),
        # full precision, odd width and odd row count, gates by token
        _norm("bn_bwd_ragged", "bn_bwd", 2999, 1237, dtype="fp32", gate=True),
        # GPT-2-XL, one large batch
        _norm("bn_bwd_gpt2xl", "bn_bwd", 131072, 1600),
    ]


def draw(rng):
    def spread(lo, hi):
        return math.exp(rng.uniform(math.log(lo), math.log(hi)))

    op = rng.choice(["glu_fwd", "glu_bwd", "bn_fwd", "bn_bwd"])
    if op.startswith("glu"):
        # the GEMMs' rule: both widths are multiples of 16
        K, F = 16 * round(spread(4, 256)), 16 * round(spread(4, 512))
        M = max(1, round(spread(1, min(32768, MAX_MKF // (K * F)))))
        if rng.random() < 0.4:
            M = max(16, M // 16 * 16)
        t = M % 16 == 0  # a transposed copy needs whole 16-byte rows
        outs = rng.choice((["hqt", "qt"] if t else ["hq"]) + ["q", "aq", "haq"] if op == "glu_fwd"
                          else (["qt", "hqt"] if t else ["hq"]) + ["h", "q"])
        return _glu(None, op, M, K, F, act=rng.choice(ACTS), outs=outs)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
    most = MAX_ELEMS // (2 if dtype == "fp32" else 1)
    N = round(spread(16, 16384))
    if rng.random() < 0.6:  # model widths are mostly multiples of 16; the rest stay as drawn
        N = max(16, N // 16 * 16)
    M = round(spread(1, min(131072, most // N)))
    return _norm(None, op, M, N, dtype=dtype, params=rng.choice(["fp32", dtype]), pad=rng.choice([0, 0, 0, 3, 16]),
                 post=rng.random() < 0.8, pre=rng.random() < 0.85, gate=rng.random() < 0.4, alpha=rng.random() < 0.5,
                 fp8=op == "bn_fwd" and dtype == "bf16" and rng.random() < 0.5)


def _glu(name, op, M, K, F, act="silu", outs="q"):
    """K: the block's width.  outs: which outputs; h the BF16 pre-activations (glu_bwd: their
    gradients), a the BF16 product, q codes, t codes transposed."""
    c = dict(op=op, M=M, K=K, F=F, act=act, outs=outs)
    return c if name is None else dict(c, name=name)


def _norm(name, op, M, N, dtype="bf16", params="fp32", post=True, pre=True, gate=False, alpha=False, fp8=False, pad=0):
    """post / pre: norm after the block, norm before the next one.  alpha: the residual's scale is a
    parameter (a gradient too)."""
    c = dict(op=op, M=M, N=N, dtype=dtype, params=params, post=post, pre=pre, gate=gate, alpha=alpha,
             fp8=fp8 and pre, pad=pad)
    return c if name is None else dict(c, name=name)


def prepare(case, seed):
    """Inputs from the seed, and the output buffers and workspace that a program keeps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def cell(v):
        return torch.full((1,), v, device="cuda")

    s = dict(case=case)
    if case["op"].startswith("glu"):
        M, K, F, fwd = case["M"], case["K"], case["F"], case["op"] == "glu_fwd"

        def codes(rows, cols, fmt, most):
            """FP8 codes of normal values whose largest is a little under the format's."""
            return normal(rows, cols).mul_(most / 6.5).clamp_(-most, most).to(fmt).view(torch.uint8)

        e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if fwd:
            # a norm's output (deviation 1) and weights of deviation K^-1/2 (margin 2 under 448): g and u about 1
            s["x_q"], s["w_q"] = codes(M, K, e4, 224.0), codes(2 * F, K, e4, 224.0)
            s["scale_x"], s["scale_w"] = cell(224.0 / 6.5), cell(224.0 / 6.5 * K ** 0.5)
        else:
            # an output gradient of deviation 1e-3 times a down-projection of deviation F^-1/2
            s["x_q"], s["w_q"] = codes(M, K, e5, 28672.0), codes(F, K, e4, 224.0)
            s["scale_x"], s["scale_w"] = cell(28672.0 / 6.5e-3), cell(224.0 / 6.5 * F ** 0.5)
            s["h"] = normal(M, 2 * F).to(torch.bfloat16)
        # the delayed scale of a step whose largest |product| was 40 (ReLU^2: 300), margin 2
        big = (300.0 if case["act"] == "relu2" else 40.0) * (1.0 if fwd else 2e-3 * max(1.0, (K / F) ** 0.5))
        s["scale_out"] = cell((448.0 if fwd else 57344.0) / (2.0 * big))
        wide = 2 * F if not fwd else F
        o, bf = case["outs"], torch.bfloat16
        s["h_out"] = empty(M, 2 * F, dtype=bf) if "h" in o else None
        s["a_out"] = empty(M, F, dtype=bf) if "a" in o else None
        s["q"] = empty(M, wide, dtype=torch.uint8) if "q" in o else None
        s["q_t"] = empty(wide, M, dtype=torch.uint8) if "t" in o else None
        s["amax"] = empty(1) if s["q"] is not None else None
        s["sat"] = empty(1, dtype=torch.int64) if s["q"] is not None else None
        return s

    M, N, T = case["M"], case["N"], TYPES[case["dtype"]]
    TW = TYPES[case["params"]]

    def rows(std):
        """[M, N] of type T, a slice of rows that are `pad` wider."""
        return normal(M, N + case["pad"]).mul_(std).to(T)[:, :N]

    s["eps"], s["post"] = EPS, case["post"]
    s["x"] = rows(0.7)  # the block's output
    s["weight"] = (1.0 + 0.1 * normal(N)).to(TW) if case["pre"] else None
    s["post_weight"] = (0.3 + 0.05 * normal(N)).to(TW)
    s["gate"] = normal(M).sigmoid_() if case["gate"] else None
    s["alpha"] = cell(0.9) if case["alpha"] else None
    if case["op"] == "bn_fwd":
        s["residual"] = rows(2.0)
        s["r_out"], s["y"] = empty(M, N, dtype=T), empty(M, N, dtype=T) if case["pre"] else None
        s["rstd"] = empty(M) if case["pre"] else None
        s["rstd_post"] = empty(M) if case["post"] else None
        if case["fp8"]:
            s["scale"] = cell(448.0 / (2.0 * 8.0))  # a previous step's maximum of 8, margin 2
            s["q"], s["amax"], s["sat"] = empty(M, N, dtype=torch.uint8), empty(1), empty(1, dtype=torch.int64)
        return s
    step = 1e-3 if T != torch.float16 else 0.5  # half precision trains with a loss scale
    s["r"] = rows(2.0)
    s["residual"] = rows(2.0) if case["alpha"] else None
    s["dy"] = rows(step) if case["pre"] else None
    s["dr"] = rows(step)
    s["rstd"] = (s["r"].float().square().mean(1) + EPS).rsqrt() if case["pre"] else None
    s["rstd_post"] = (s["x"].float().square().mean(1) + EPS).rsqrt() if case["post"] else None
    s["dresidual"], s["dx"] = empty(M, N, dtype=T), empty(M, N, dtype=T)
    s["dweight"] = empty(N) if case["pre"] else None
    s["dpost_weight"] = empty(N)
    s["dgate"] = empty(M) if case["gate"] else None
    s["dalpha"] = empty(1) if case["alpha"] else None
    # partial column sums: at most 1024 rows of two sums a column and four cells
    s["workspace"] = torch.empty(1024 * (8 * N + 16), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from quantize_fp8_gemm_gb300 import binding as B
    op = s["case"]["op"]
    if op.startswith("glu"):
        act = {"identity": B.ACT_IDENTITY, "relu": B.ACT_RELU, "relu2": B.ACT_RELU2, "silu": B.ACT_SILU,
               "gelu": B.ACT_GELU}[s["case"]["act"]]
        if op == "glu_fwd":
            B.fp8_glu_fwd(s["x_q"], s["w_q"], s["scale_x"], s["scale_w"], act=act, h_out=s["h_out"],
                          act_out=s["a_out"], scale_a=s["scale_out"], a_q=s["q"], a_q_t=s["q_t"], amax_out=s["amax"],
                          sat_count=s["sat"], status=s["status"])
        else:
            B.fp8_gemm_dgrad_glu(s["x_q"], s["w_q"], s["scale_x"], s["scale_w"], s["h"], act=act, dh=s["h_out"],
                                 scale_dh=s["scale_out"], dh_q=s["q"], dh_q_t=s["q_t"], amax_out=s["amax"],
                                 sat_count=s["sat"], status=s["status"])
        return _glu_outputs(s, s["h_out"], s["a_out"], s["q"], s["q_t"], s["amax"], s["sat"])
    if op == "bn_fwd":
        codes = dict(scale=s["scale"], q_out=s["q"], amax_out=s["amax"], sat_count=s["sat"]) if s["case"]["fp8"] else {}
        B.block_norm_fwd(s["x"], s["weight"], s["y"], eps=s["eps"], rstd=s["rstd"], residual=s["residual"],
                         alpha=s["alpha"], gate=s["gate"], post_weight=s["post_weight"], post_norm=s["post"],
                         rstd_post=s["rstd_post"], r_out=s["r_out"], **codes)
        return _fwd_outputs(s, s["r_out"], s["y"], s["rstd"], s["rstd_post"], s.get("q"), s.get("amax"), s.get("sat"))
    B.block_norm_bwd(s["dy"], s["r"], s["rstd"], s["weight"], dr=s["dr"], x=s["x"], residual=s["residual"],
                     alpha=s["alpha"], gate=s["gate"], post_weight=s["post_weight"], post_norm=s["post"],
                     rstd_post=s["rstd_post"], dresidual=s["dresidual"], dx=s["dx"], dweight=s["dweight"],
                     dpost_weight=s["dpost_weight"], dgate=s["dgate"], dalpha=s["dalpha"], workspace=s["workspace"])
    return _kept(dresidual=s["dresidual"], dx=s["dx"], dweight=s["dweight"], dpost_weight=s["dpost_weight"],
                 dgate=s["dgate"], dalpha=s["dalpha"])


def _kept(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _glu_outputs(s, h, a, q, q_t, amax, sat):
    fmt = torch.float8_e4m3fn if s["case"]["op"] == "glu_fwd" else torch.float8_e5m2
    return _kept(h=h, a=a, q=None if q is None else q.view(fmt), q_t=None if q_t is None else q_t.view(fmt),
                 amax=amax, sat=sat)


def _fwd_outputs(s, r, y, rstd, rstd_post, q, amax, sat):
    return _kept(r=r, y=y, rstd=rstd, rstd_post=rstd_post, q=None if q is None else q.view(torch.float8_e4m3fn),
                 amax=amax, sat=sat)


# ------------------------------------------------------------------------------------------- plain form
_GELU_C, _GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, g, grad):
    """act(g), or with grad its derivative."""
    if name == "identity":
        return torch.ones_like(g) if grad else g
    if name == "relu":
        return (g > 0).float() if grad else torch.where(g > 0, g, torch.zeros_like(g))
    if name == "relu2":
        p = torch.where(g > 0, g, torch.zeros_like(g))
        return 2.0 * p if grad else p * p
    # SiLU g sigma(g); GELU's tanh form 0.5 g (1 + tanh z) = g sigma(2 z)
    z = g if name == "silu" else 2.0 * _GELU_C * (g + _GELU_B * g * g * g)
    sig = 1.0 / (1.0 + torch.exp(-z))
    if not grad:
        return g * sig
    dz = 1.0 if name == "silu" else 2.0 * _GELU_C * (1.0 + 3.0 * _GELU_B * g * g)
    return sig + g * sig * (1.0 - sig) * dz


def _codes(s, v):
    """The outputs that hang on codes of the rounded values v."""
    fwd = s["case"]["op"] != "glu_bwd"
    scaled = v.float() * (s["scale"] if "scale" in s else s["scale_out"])
    most = 448.0 if fwd else 57344.0
    q = scaled.clamp(-most, most).to(torch.float8_e4m3fn if fwd else torch.float8_e5m2).view(torch.uint8)
    return q, v.float().abs().max().reshape(1), (scaled.abs() > most).sum().reshape(1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op.startswith("glu"):
        fwd, F, o, bf = op == "glu_fwd", c["F"], c["outs"], torch.bfloat16
        x = s["x_q"].view(torch.float8_e4m3fn if fwd else torch.float8_e5m2).float()
        prod = (x @ s["w_q"].view(torch.float8_e4m3fn).float().t()) * (1.0 / (s["scale_x"] * s["scale_w"]))
        if fwd:
            h, v = prod, (_act(c["act"], prod[:, :F], False) * prod[:, F:]).to(bf)
        else:
            g, u = s["h"][:, :F].float(), s["h"][:, F:].float()
            h = v = torch.cat([prod * u * _act(c["act"], g, True), prod * _act(c["act"], g, False)], 1).to(bf)
        q = q_t = amax = sat = None
        if "q" in o:
            q, amax, sat = _codes(s, v)
            q_t = q.t().contiguous() if "t" in o else None
        return _glu_outputs(s, h.to(bf) if "h" in o else None, v if "a" in o else None, q, q_t, amax, sat)

    T, N = TYPES[c["dtype"]], c["N"]
    x, wp = s["x"].float(), s["post_weight"].float()
    alpha = s["alpha"] if c["alpha"] else 1.0
    gate = s["gate"][:, None] if c["gate"] else 1.0
    if op == "bn_fwd":
        rstd_post = rstd = y = q = amax = sat = None
        if c["post"]:
            rstd_post = 1.0 / torch.sqrt(x.square().sum(1) / N + s["eps"])
            x = x * rstd_post[:, None]
        stored = (alpha * s["residual"].float() + gate * (x * wp)).to(T)
        if c["pre"]:
            r = stored.float()
            rstd = 1.0 / torch.sqrt(r.square().sum(1) / N + s["eps"])
            y = (r * rstd[:, None] * s["weight"].float()).to(T)
        if c["fp8"]:
            q, amax, sat = _codes(s, y)
        return _fwd_outputs(s, stored, y, rstd, rstd_post, q, amax, sat)
    dr, dweight, dgate, dalpha = s["dr"].float(), None, None, None
    if c["pre"]:
        dy, rhat = s["dy"].float(), s["r"].float() * s["rstd"][:, None]
        dweight = (dy * rhat).sum(0)
        g = dy * s["weight"].float()
        dr = dr + (g - rhat * ((g * rhat).sum(1, keepdim=True) / N)) * s["rstd"][:, None]
    if c["alpha"]:
        dalpha = (dr * s["residual"].float()).sum().reshape(1)
    if c["post"]:
        x = x * s["rstd_post"][:, None]
    t = dr * wp
    along = (t * x).sum(1)
    dx = (t - x * (along[:, None] / N)) * s["rstd_post"][:, None] if c["post"] else t
    if c["gate"]:
        dgate = along
    return _kept(dresidual=(alpha * dr).to(T), dx=(gate * dx).to(T), dweight=dweight,
                 dpost_weight=(gate * dr * x).sum(0), dgate=dgate, dalpha=dalpha)


def work(case):
    if case["op"].startswith("glu"):
        M, K, F, o, fwd = case["M"], case["K"], case["F"], case["outs"], case["op"] == "glu_fwd"
        wide = F if fwd else 2 * F
        out = M * (4 * F * ("h" in o) + 2 * F * ("a" in o) + wide * (("q" in o) + ("t" in o)))
        return {"bytes": M * K + (2 if fwd else 1) * F * K + (0 if fwd else 4 * M * F) + out,
                "flops": (4.0 if fwd else 2.0) * M * K * F + 20.0 * M * F}
    M, N = case["M"], case["N"]
    es, ps = (2 if case["dtype"] != "fp32" else 4), (2 if case["params"] != "fp32" else 4)
    if case["op"] == "bn_fwd":
        return {"bytes": M * N * ((3 + case["pre"]) * es + case["fp8"]) + 4 * M * (case["post"] + case["pre"] + case["gate"])
                + N * ps * (1 + case["pre"]), "flops": M * N * (4.0 + 2 * case["post"] + 4 * case["pre"])}
    tensors = 4 + 2 * case["pre"] + case["alpha"]
    return {"bytes": M * N * tensors * es + 4 * M * (case["post"] + case["pre"] + 2 * case["gate"])
            + N * (ps + 4) * (1 + case["pre"]), "flops": M * N * (8.0 + 10 * case["pre"] + 4 * case["post"])}


# --------------------------------------------------------------------------------- definition in 64 bits
def _exact_act(name, g):
    """(act(g), act'(g)) from the definitions, by tanh."""
    if name == "identity":
        return g, torch.ones_like(g)
    if name.startswith("relu"):
        p = g.clamp(min=0.0)
        return (p, torch.heaviside(g, torch.zeros_like(g))) if name == "relu" else (p.pow(2), p.mul(2.0))
    if name == "silu":
        th = torch.tanh(g / 2)
        return (g + g * th) / 2, (1 + th) / 2 + g * (1 - th * th) / 4
    inner = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3)))
    slope = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g.pow(2))
    return g / 2 * (1 + inner), (1 + inner) / 2 + g / 2 * (1 - inner.pow(2)) * slope


def exact(case, seed):
    """What ``run`` returns, from the definitions in float64, by blocks of rows.  The stream r, which is
    defined as rounded and feeds other outputs, is rounded; so are the values whose codes and largest
    magnitude are outputs, and the codes are those of the format."""
    s = prepare(case, seed)
    M, out = case["M"], {}

    def put(name, lo, hi, v, turned=False):
        if name not in out:
            out[name] = torch.empty((v.shape[1], M) if turned else (M,) + v.shape[1:], dtype=torch.float64, device="cuda")
        if turned:
            out[name][:, lo:hi] = v.T
        else:
            out[name][lo:hi] = v

    def scalar(v):
        return torch.tensor([v], dtype=torch.float64, device="cuda")

    def put_codes(lo, hi, v, scale, most, fmt, turned):
        """The codes of v, a value already rounded to its type, and its largest magnitude so far."""
        coded = torch.clamp(v.float() * scale, -most, most).to(fmt).double()
        put("q", lo, hi, coded)
        if turned:
            put("q_t", lo, hi, coded, True)
        return float(v.abs().max())

    if case["op"].startswith("glu"):
        K, F, o, fwd = case["K"], case["F"], case["outs"], case["op"] == "glu_fwd"
        w = s["w_q"].view(torch.float8_e4m3fn).double() / s["scale_w"].double()
        most, big = (448.0 if fwd else 57344.0), 0.0
        step = max(1, (1 << 25) // F)
        for lo in range(0, M, step):
            hi = min(M, lo + step)
            x = s["x_q"][lo:hi].view(torch.float8_e4m3fn if fwd else torch.float8_e5m2).double() / s["scale_x"].double()
            prod = torch.einsum("mk,fk->mf", x, w)
            if fwd:
                g, u = prod.split(F, dim=1)
                v = _exact_act(case["act"], g)[0] * u
                if "h" in o:
                    put("h", lo, hi, prod)
                if "a" in o:
                    put("a", lo, hi, v)
            else:
                g, u = s["h"][lo:hi].double().split(F, dim=1)
                f, df = _exact_act(case["act"], g)
                v = torch.hstack([prod * df * u, prod * f])
                if "h" in o:
                    put("h", lo, hi, v)
            if "q" in o:
                big = max(big, put_codes(lo, hi, v.to(torch.bfloat16), s["scale_out"], most,
                                         torch.float8_e4m3fn if fwd else torch.float8_e5m2, "t" in o))
        if "q" in o:
            out["amax"], out["sat"] = scalar(big), None
        return out

    N, T = case["N"], TYPES[case["dtype"]]
    step = max(1, (1 << 24) // N)
    wp, w = s["post_weight"].double(), s["weight"].double() if case["pre"] else None
    alpha = float(s["alpha"]) if case["alpha"] else 1.0
    sums = {}
    for lo in range(0, M, step):
        hi = min(M, lo + step)

        def rows_of(name):
            return s[name][lo:hi].double()

        x = rows_of("x")
        gate = rows_of("gate")[:, None] if case["gate"] else torch.ones(hi - lo, 1, dtype=torch.float64, device="cuda")
        if case["op"] == "bn_fwd":
            if case["post"]:
                rms = (torch.linalg.vector_norm(x, dim=1) ** 2 / N + EPS) ** 0.5
                put("rstd_post", lo, hi, 1 / rms)
                x = x / rms[:, None]
            r = torch.addcmul(rows_of("residual") * alpha, x * gate, wp)
            put("r", lo, hi, r)
            if not case["pre"]:
                continue
            r = r.to(T).double()
            rms = (torch.linalg.vector_norm(r, dim=1) ** 2 / N + EPS) ** 0.5
            y = r / rms[:, None] * w
            put("rstd", lo, hi, 1 / rms), put("y", lo, hi, y)
            if case["fp8"]:
                big = put_codes(lo, hi, y.to(T), s["scale"], 448.0, torch.float8_e4m3fn, False)
                sums["amax"] = max(sums.get("amax", 0.0), big)
            continue
        dr = rows_of("dr")
        if case["pre"]:
            dy, r, rstd = rows_of("dy"), rows_of("r"), rows_of("rstd")[:, None]
            sums["dweight"] = sums.get("dweight", 0.0) + torch.einsum("mn,mn,m->n", dy, r, rstd[:, 0])
            g = dy * w
            dr = dr + rstd * g - r * rstd.pow(3) * torch.einsum("mn,mn->m", g, r)[:, None] / N
        put("dresidual", lo, hi, dr * alpha)
        if case["alpha"]:
            sums["dalpha"] = sums.get("dalpha", 0.0) + float(torch.einsum("mn,mn->", dr, rows_of("residual")))
        k = rows_of("rstd_post")[:, None] if case["post"] else torch.ones_like(gate)
        sums["dpost_weight"] = sums.get("dpost_weight", 0.0) + torch.einsum("mn,mn,m->n", dr, x, (gate * k)[:, 0])
        dot = torch.einsum("mn,mn,n->m", dr, x, wp)[:, None]
        dx = dr * wp * k - (x * k.pow(3) * dot / N if case["post"] else 0.0)
        put("dx", lo, hi, dx * gate)
        if case["gate"]:
            put("dgate", lo, hi, (dot * k)[:, 0])
    for name, v in sums.items():
        out[name] = scalar(v) if name in ("amax", "dalpha") else v
    if "amax" in sums:
        out["sat"] = None
    return out
