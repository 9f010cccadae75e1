"""Cases of the operators around the FP8 MLP: layer norm and dropout, both directions.

One transformer sub-layer is  out = x + dropout(mlp(layer_norm(x))).  Its matrix products are the
framework's FP8 GEMMs; what stands around them is measured here:

    layer_norm_fwd   statistics, normalised output, optionally the E4M3 codes the up-projection
                     reads, and optionally the dropout and residual addition that come before it
    layer_norm_bwd   the input's gradient with the residual's added, optionally the dropped
                     branch's gradient, and the column sums of the weight's and bias's gradients
    dropout_fwd      dropout with the residual added;  dropout_bwd its gradient

A dropout mask is never stored: element (i, j) is dropped when word j % 4 of Philox4x32-10 (Salmon et
al., "Parallel random numbers: as easy as 1, 2, 3", 2011) at the counter (j / 4, i, offset low, offset
high) under the key (seed low, seed high) is below round(p 2^32).  Seed and offset are inputs.

``run`` computes plainly, in float32, with elementary torch operations; with ``own`` set it calls the
framework.  The residual stream r = residual + dropout(x) is an output in the activations' type, and
the layer norm is that of the r which is stored: so its gradient, taken from the stored r, is the
gradient of what was computed.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAX_ELEMS = 131072 * 1600  # elements of the largest listed case
MAX_PARTIALS = 1024


def listed():
    return [
        # the smallest workload of the framework's own tests: a call's latency
        _case("ln_fwd_tiny", "ln_fwd", 64, 64),
        # GPT-2-small, one batch: the pre-MLP norm, its E4M3 codes going into the up-projection
        _case("ln_fwd_gpt2s_fp8", "ln_fwd", 8192, 768, fp8=True),
        # odd width, half precision, rows cut out of a wider buffer
        _case("ln_fwd_ragged", "ln_fwd", 5003, 1001, dtype="fp16", params="fp16", pad=6),
        # GPT-2-XL, one large batch: dropout, residual, norm and codes in one pass between two layers
        _case("drop_add_ln_fwd_gpt2xl", "ln_fwd", 131072, 1600, residual=True, p=0.1, fp8=True),
        # the tiny workload's gradient
        _case("ln_bwd_tiny", "ln_bwd", 64, 64, residual=True),
        # GPT-2-small, one batch: the norm's gradient with the residual's added
        _case("ln_bwd_gpt2s", "ln_bwd", 8192, 768, residual=True),
        # full precision, odd width and odd row count
        _case("ln_bwd_ragged", "ln_bwd", 2999, 1237, dtype="fp32"),
        # GPT-2-XL, one large batch: the whole gradient between two layers, the dropped branch's included
        _case("drop_add_ln_bwd_gpt2xl", "ln_bwd", 131072, 1600, residual=True, p=0.1),
        # GPT-2-small, large batch: the end of a sub-layer
        _case("dropout_fwd_gpt2s_batch", "drop_fwd", 65536, 768, residual=True, p=0.1),
        # a few tokens, odd width, no residual
        _case("dropout_fwd_few", "drop_fwd", 37, 1025, dtype="fp32", p=0.25),
        # the outlier workload's width: the gradient at the end of a sub-layer
        _case("dropout_bwd_outlier", "drop_bwd", 16384, 1024, p=0.1),
        # half precision, odd width
        _case("dropout_bwd_ragged", "drop_bwd", 4097, 333, dtype="fp16", p=0.5),
    ]


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_fwd", "ln_bwd", "ln_bwd", "drop_fwd", "drop_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
    most = MAX_ELEMS // (2 if dtype == "fp32" else 1)
    N = round(math.exp(rng.uniform(math.log(16), math.log(16384))))
    if rng.random() < 0.6:  # model widths are mostly multiples of 16; the rest stay as drawn
        N = max(16, N // 16 * 16)
    M = round(math.exp(rng.uniform(0.0, math.log(min(131072, most // N)))))
    drop = op.startswith("drop") or rng.random() < 0.4
    return _case(None, op, M, N, dtype=dtype, params=rng.choice(["fp32", dtype]),
                 pad=rng.choice([0, 0, 0, 3, 16]), residual=op != "drop_bwd" and (drop or rng.random() < 0.5),
                 p=round(rng.uniform(0.01, 0.6), 3) if drop else 0.0,
                 fp8=op == "ln_fwd" and dtype == "bf16" and rng.random() < 0.5)


def _case(name, op, M, N, dtype="bf16", params="fp32", residual=False, p=0.0, fp8=False, pad=0):
    c = dict(op=op, M=M, N=N, dtype=dtype, params=params, residual=residual, p=p, fp8=fp8, pad=pad)
    return c if name is None else dict(c, name=name)


def prepare(case, seed):
    """Inputs from the seed, and the output buffers and workspace that a training program keeps."""
    M, N, T, dev = case["M"], case["N"], TYPES[case["dtype"]], "cuda"
    TW = TYPES[case["params"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def rows(std):
        """[M, N] of type T, a slice of rows that are `pad` wider."""
        return normal(M, N + case["pad"]).mul_(std).to(T)[:, :N]

    s = dict(case=case, eps=EPS, p=case["p"])
    # the 64-bit seed and offset of the generator, as a training step keeps them on the device
    s["rng"] = torch.randint(-(1 << 62), 1 << 62, (2,), generator=gen, device=dev, dtype=torch.int64)
    if case["op"].startswith("ln"):
        s["weight"] = (1.0 + 0.1 * normal(N)).to(TW)
        s["bias"] = (0.02 * normal(N)).to(TW)
    if case["op"] == "ln_fwd":
        s["x"] = rows(1.0)
        s["residual"] = rows(2.0) if case["residual"] else None
        s["y"] = torch.empty(M, N, dtype=T, device=dev)
        s["r_out"] = torch.empty(M, N, dtype=T, device=dev) if case["residual"] or case["p"] else None
        s["mean"], s["rstd"] = torch.empty(M, device=dev), torch.empty(M, device=dev)
        if case["fp8"]:
            # the delayed scale: format maximum over margin 2 times a previous step's maximum of 6
            s["scale"] = torch.full((1,), 448.0 / (2.0 * 6.0), device=dev)
            s["q_out"] = torch.empty(M, N, dtype=torch.uint8, device=dev)
            s["amax_out"] = torch.zeros(1, device=dev)
            s["sat_count"] = torch.zeros(1, dtype=torch.int64, device=dev)
    elif case["op"] == "ln_bwd":
        s["x"] = rows(2.0)
        s["dy"] = rows(1e-3 if T != torch.float16 else 0.5)  # half precision trains with a loss scale
        s["dresidual"] = rows(1e-3 if T != torch.float16 else 0.5) if case["residual"] else None
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = 1.0 / ((x - s["mean"][:, None]).square().mean(1) + EPS).sqrt()
        s["dx"] = torch.empty(M, N, dtype=T, device=dev)
        s["dbranch"] = torch.empty(M, N, dtype=T, device=dev) if case["p"] else None
        s["dweight"], s["dbias"] = torch.empty(N, device=dev), torch.empty(N, device=dev)
        # partial column sums: at most this many rows of 2 N floats
        s["workspace"] = torch.empty(MAX_PARTIALS * 8 * N, dtype=torch.uint8, device=dev)
    elif case["op"] == "drop_fwd":
        s["x"] = rows(1.0)
        s["residual"] = rows(2.0) if case["residual"] else None
        s["y"] = torch.empty(M, N, dtype=T, device=dev)
    else:
        s["dy"] = rows(1e-3 if T != torch.float16 else 0.5)
        s["dx"] = torch.empty(M, N, dtype=T, device=dev)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from quantize_fp8_gemm_gb300 import binding as B
    op, p = s["case"]["op"], s["p"]
    if op == "ln_fwd":
        if s["case"]["fp8"]:
            B.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["y"], eps=s["eps"], mean=s["mean"], rstd=s["rstd"],
                             residual=s["residual"], r_out=s["r_out"], p=p, rng=s["rng"], fmt=B.E4M3,
                             scale=s["scale"], q_out=s["q_out"], amax_out=s["amax_out"], sat_count=s["sat_count"])
        else:
            B.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["y"], eps=s["eps"], mean=s["mean"], rstd=s["rstd"],
                             residual=s["residual"], r_out=s["r_out"], p=p, rng=s["rng"])
        return _fwd_outputs(s, s["y"], s["mean"], s["rstd"], s["r_out"], s.get("q_out"), s.get("amax_out"),
                            s.get("sat_count"))
    if op == "ln_bwd":
        B.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], s["dx"], dresidual=s["dresidual"],
                         dweight=s["dweight"], dbias=s["dbias"], workspace=s["workspace"], p=p, rng=s["rng"],
                         dbranch=s["dbranch"])
        return _bwd_outputs(s, s["dx"], s["dweight"], s["dbias"], s["dbranch"])
    if op == "drop_fwd":
        B.dropout_fwd(s["x"], s["y"], p, s["rng"], residual=s["residual"])
        return {"y": s["y"]}
    B.dropout_bwd(s["dy"], s["dx"], p, s["rng"])
    return {"dx": s["dx"]}


def _fwd_outputs(s, y, mean, rstd, r, q, amax, sat):
    out = {"y": y, "mean": mean, "rstd": rstd}
    if r is not None:
        out["r"] = r
    if s["case"]["fp8"]:
        out.update(q=q.view(torch.float8_e4m3fn), amax=amax, sat=sat)
    return out


def _bwd_outputs(s, dx, dweight, dbias, dbranch):
    out = {"dx": dx, "dweight": dweight, "dbias": dbias}
    if dbranch is not None:
        out["dbranch"] = dbranch
    return out


# ------------------------------------------------------------------------------------------- plain form
_LOW = 0xFFFFFFFF


def _mul_hi_lo(a, m):
    """(high, low) 32-bit words of a * m, a an int64 tensor below 2^32."""
    prod = a * m  # the low 64 bits, whatever the sign
    return (prod >> 32) & _LOW, prod & _LOW


def _keep(rng, M, N, p):
    """The keep mask [M, N]."""
    quads = (N + 3) // 4
    key, off = rng[0], rng[1]
    c0 = torch.arange(quads, device=rng.device)[None, :]
    c1 = torch.arange(M, device=rng.device)[:, None]
    c2, c3 = off & _LOW, (off >> 32) & _LOW
    k0, k1 = key & _LOW, (key >> 32) & _LOW
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    below = round(p * 4294967296.0)
    kept = torch.stack([w.expand(M, quads) >= below for w in (c0, c1, c2, c3)], dim=2)
    return kept.reshape(M, 4 * quads)[:, :N]


def _dropped(x, s):
    """keep ? x / (1 - p) : 0 in float32."""
    M, N = x.shape
    scaled = x.float() * (1.0 / (1.0 - s["p"]))
    return torch.where(_keep(s["rng"], M, N, s["p"]), scaled, torch.zeros_like(scaled))


def _run_plain(s):
    op, T = s["case"]["op"], TYPES[s["case"]["dtype"]]
    if op == "ln_fwd":
        r, stored = s["x"], None
        if s["residual"] is not None or s["p"]:
            r = _dropped(s["x"], s) if s["p"] else s["x"].float()
            if s["residual"] is not None:
                r = s["residual"].float() + r
            r = stored = r.to(T)
        r = r.float()
        mean = r.sum(1) / r.shape[1]
        dev = r - mean[:, None]
        rstd = 1.0 / torch.sqrt(dev.square().sum(1) / r.shape[1] + s["eps"])
        y = (dev * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(T)
        q = amax = sat = None
        if s["case"]["fp8"]:
            v = y.float() * s["scale"]
            q = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            amax = y.float().abs().max().reshape(1)
            sat = (v.abs() > 448.0).sum().reshape(1)
        return _fwd_outputs(s, y, mean, rstd, stored, q, amax, sat)
    if op == "ln_bwd":
        N = s["x"].shape[1]
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dweight, dbias = (dy * xhat).sum(0), dy.sum(0)
        g = dy * s["weight"].float()
        c1, c2 = g.sum(1, keepdim=True) / N, (g * xhat).sum(1, keepdim=True) / N
        dr = (g - c1 - xhat * c2) * s["rstd"][:, None]
        if s["dresidual"] is not None:
            dr = dr + s["dresidual"].float()
        dbranch = _dropped(dr, s).to(T) if s["p"] else None
        return _bwd_outputs(s, dr.to(T), dweight, dbias, dbranch)
    if op == "drop_fwd":
        d = _dropped(s["x"], s)
        return {"y": (s["residual"].float() + d if s["residual"] is not None else d).to(T)}
    return {"dx": _dropped(s["dy"], s).to(T)}


def work(case):
    M, N = case["M"], case["N"]
    es, ps = (2 if case["dtype"] != "fp32" else 4), (2 if case["params"] != "fp32" else 4)
    mn, drop = M * N, 40.0 / 4 if case["p"] else 0.0  # one generator block of about 40 operations for four elements
    if case["op"] == "ln_fwd":
        tensors = 2 + bool(case["residual"]) + bool(case["residual"] or case["p"])
        return {"bytes": mn * (tensors * es + bool(case["fp8"])) + 8 * M + 2 * N * ps,
                "flops": mn * (8.0 + bool(case["residual"]) + 2 * bool(case["fp8"]) + drop)}
    if case["op"] == "ln_bwd":
        tensors = 3 + bool(case["residual"]) + bool(case["p"])
        return {"bytes": mn * tensors * es + 8 * M + N * ps + 8 * N, "flops": mn * (14.0 + bool(case["residual"]) + drop)}
    tensors = 2 + bool(case["residual"])
    return {"bytes": mn * tensors * es, "flops": mn * (1.0 + bool(case["residual"]) + drop)}


# --------------------------------------------------------------------------------- definition in 64 bits
def _exact_keep(seed, offset, row0, m, N, p):
    """Rows row0 .. row0 + m of the mask.  Written from the generator's definition on 16-bit halves, so
    that no product passes 2^33: a way of its own to the same bits as the plain form's."""
    quads = -(-N // 4)
    j = torch.arange(m * quads, device="cuda")
    ctr = [j % quads, j // quads + row0, torch.full_like(j, offset & _LOW), torch.full_like(j, offset >> 32 & _LOW)]
    key = [seed & _LOW, seed >> 32 & _LOW]

    def times(a, c):
        al, ah, cl, ch = a & 0xFFFF, a >> 16, c & 0xFFFF, c >> 16
        mid = al * ch + (al * cl >> 16)
        mid2 = ah * cl + (mid & 0xFFFF)
        return ah * ch + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (al * cl & 0xFFFF)

    for r in range(10):
        k = [(key[0] + r * 0x9E3779B9) & _LOW, (key[1] + r * 0xBB67AE85) & _LOW]
        (ha, la), (hb, lb) = times(ctr[0], 0xD2511F53), times(ctr[2], 0xCD9E8D57)
        ctr = [hb ^ ctr[1] ^ k[0], lb, ha ^ ctr[3] ^ k[1], la]
    limit = int(round(p * 2 ** 32))
    keep = torch.empty(m, quads, 4, dtype=torch.bool, device="cuda")
    for w in range(4):
        keep[:, :, w] = (ctr[w] >= limit).view(m, quads)
    return keep.view(m, -1)[:, :N]


def exact(case, seed):
    """What ``run`` returns, from the definitions in float64, by blocks of rows.  A value that is defined
    as rounded and feeds another output (r) is rounded; codes have the unrounded product as their value."""
    s = prepare(case, seed)
    M, N, p = case["M"], case["N"], case["p"]
    T, op = TYPES[case["dtype"]], case["op"]
    gseed, goff = (int(v) for v in s["rng"].tolist())
    step = max(1, (1 << 24) // N)
    out, sums = {}, {}

    def rows_of(name, lo, hi):
        return s[name][lo:hi].double()

    def put(name, lo, hi, v):
        if name not in out:
            out[name] = torch.empty((M,) + v.shape[1:], dtype=torch.float64, device="cuda")
        out[name][lo:hi] = v

    def masked(v, lo, hi):
        return v / (1.0 - p) * _exact_keep(gseed, goff, lo, hi - lo, N, p)

    w = s["weight"].double() if "weight" in s else None
    for lo in range(0, M, step):
        hi = min(M, lo + step)
        if op == "ln_fwd":
            r = rows_of("x", lo, hi)
            if p:
                r = masked(r, lo, hi)
            if case["residual"]:
                r = r + rows_of("residual", lo, hi)
            if p or case["residual"]:
                put("r", lo, hi, r)
                r = r.to(T).double()
            var, mean = torch.var_mean(r, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["bias"].double(), (r - mean[:, None]) * rstd[:, None], w)
            put("y", lo, hi, y), put("mean", lo, hi, mean), put("rstd", lo, hi, rstd)
            if case["fp8"]:
                v = y * s["scale"].double()
                put("q", lo, hi, torch.clamp(v, -448.0, 448.0))
                sums["amax"] = max(sums.get("amax", 0.0), float(y.abs().max()))
        elif op == "ln_bwd":
            dy = rows_of("dy", lo, hi)
            xhat = (rows_of("x", lo, hi) - s["mean"][lo:hi, None].double()) * s["rstd"][lo:hi, None].double()
            sums["dweight"] = sums.get("dweight", 0.0) + torch.einsum("mn,mn->n", dy, xhat)
            sums["dbias"] = sums.get("dbias", 0.0) + dy.sum(0)
            g = dy * w
            along = xhat * (g * xhat).mean(1, keepdim=True) + g.mean(1, keepdim=True)
            dr = (g - along) * s["rstd"][lo:hi, None].double()
            if case["residual"]:
                dr = dr + rows_of("dresidual", lo, hi)
            put("dx", lo, hi, dr)
            if p:
                put("dbranch", lo, hi, masked(dr, lo, hi))
        elif op == "drop_fwd":
            y = masked(rows_of("x", lo, hi), lo, hi)
            put("y", lo, hi, y + rows_of("residual", lo, hi) if case["residual"] else y)
        else:
            put("dx", lo, hi, masked(rows_of("dy", lo, hi), lo, hi))
    if "amax" in sums:
        out["amax"], out["sat"] = torch.tensor([sums["amax"]], dtype=torch.float64, device="cuda"), None
    for name in ("dweight", "dbias"):
        if name in sums:
            out[name] = sums[name]
    return out
