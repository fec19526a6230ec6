"""Cases that measure the decode-side operators: RMS norm with the residual's
addition (bfloat16 or MXFP8 output), products with 4-bit weights for a few
tokens, and a whole MoE layer for a few tokens (bfloat16 or 4-bit weights).

Each operator also stands here in its plain form (elementary torch operations
in float32), which runs without the library; with ``own`` set, ``run`` makes
the library's calls instead. ``exact`` evaluates the definitions in float64.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    """Sizes are those of the library's own workloads: decode (H=7168, E=256,
    top-8, I=2048), mid (H=2048, E=128, top-8, I=768), prefill (H=4096, E=8,
    top-2, I=14336), skewed (H=2880, E=32, top-4, I=2880)."""
    return [
        # the norm before the MoE layer of a decode step: latency
        dict(name="norm decode", op="norm", T=16, H=7168, out="bf16"),
        # the same norm over a prefill chunk: bandwidth
        dict(name="norm prefill", op="norm", T=8192, H=4096, out="bf16"),
        # an odd chunk, output for an 8-bit expert GEMM alone
        dict(name="norm mxfp8 odd", op="norm", T=1023, H=2880, out="mxfp8"),
        # 8 bits for the GEMM and bfloat16 for the router
        dict(name="norm mxfp8 both", op="norm", T=4096, H=2048, out="both"),
        # one token through a small projection: the smallest call
        dict(name="gemv smallest", op="gemv", T=1, N=2048, K=768, fmt="mxfp4", out="bf16"),
        # a decode batch through a dense projection
        dict(name="gemv decode", op="gemv", T=16, N=4096, K=7168, fmt="nvfp4", out="bf16"),
        # the most tokens, odd widths, float32 results (logits)
        dict(name="gemv full batch", op="gemv", T=32, N=5760, K=2880, fmt="mxfp4", out="f32"),
        # a wide projection, an odd number of tokens
        dict(name="gemv wide", op="gemv", T=7, N=28672, K=4096, fmt="nvfp4", out="bf16"),
        # one user's token through a layer of small experts: latency
        dict(name="layer one token", op="layer", T=1, H=2048, E=128, k=8, I=768, renorm=True, fmt="bf16"),
        # a decode batch over many large experts: the largest
        dict(name="layer decode", op="layer", T=16, H=7168, E=256, k=8, I=2048, renorm=False, fmt="bf16"),
        # a small batch, 4-bit weights with a scale per 32, most experts hit
        dict(name="layer mxfp4", op="layer", T=8, H=2880, E=32, k=4, I=2880, renorm=True, fmt="mxfp4"),
        # the most tokens, few wide experts, 4-bit weights with a scale per 16
        dict(name="layer nvfp4 wide", op="layer", T=32, H=4096, E=8, k=2, I=14336, renorm=True, fmt="nvfp4"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["norm", "gemv", "layer", "layer"])
    while True:
        if op == "norm":
            c = dict(op=op, out=rng.choice(["bf16", "mxfp8", "both"]), T=_log(rng, 1, 8192))
            c["H"] = _mult(rng, 256, 8192, 8 if c["out"] == "bf16" else 32)
            if c["T"] * c["H"] <= 8192 * 4096:
                return c
        elif op == "gemv":
            c = dict(op=op, T=_log(rng, 1, 32), N=_log(rng, 64, 28672), K=_mult(rng, 256, 8192, 32),
                     fmt=rng.choice(["nvfp4", "mxfp4"]), out=rng.choice(["bf16", "f32"]))
            if c["N"] * c["K"] <= 28672 * 4096:
                return c
        else:
            c = dict(op=op, fmt=rng.choice(["bf16", "nvfp4", "mxfp4"]), T=_log(rng, 1, 32), E=_log(rng, 8, 256))
            m = 8 if c["fmt"] == "bf16" else 32
            c.update(k=rng.randint(1, 8), H=_mult(rng, 512, 7168, m), I=_mult(rng, 256, 14336, m),
                     renorm=rng.random() < 0.5)
            weights = c["E"] * c["H"] * c["I"] * 3
            if weights <= 2 * 10 ** 9 and min(c["T"] * c["k"], c["E"]) * c["H"] * c["I"] <= 5 * 10 ** 8:
                return c


def work(c):
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        out = {"bf16": 2.0, "mxfp8": 1 + 1 / 32, "both": 3 + 1 / 32}[c["out"]]
        return {"bytes": n * (6 + out) + 2 * c["H"], "flops": 8 * n}
    if c["op"] == "gemv":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": N * K * (0.5 + 1 / BLOCK[c["fmt"]]) + 2 * T * K + T * N * (2 if c["out"] == "bf16" else 4),
                "flops": 2 * T * N * K}
    T, H, E, k, I = (c[n] for n in ("T", "H", "E", "k", "I"))
    distinct = E * (1 - (1 - k / E) ** T)   # expected over routings: each token takes k of E
    per = 2.0 if c["fmt"] == "bf16" else 0.5 + 1 / BLOCK[c["fmt"]]
    return {"bytes": distinct * 3 * H * I * per + 4 * T * H + 4 * T * E + 8 * T * k, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)


def _quantize(w, fmt):
    """float32 weights [..., n] -> (codes [..., n/2], scales [..., n/block], g)
    in the library's 4-bit formats, g per leading matrix (1 for MXFP4)."""
    blocks = w.unflatten(-1, (-1, BLOCK[fmt]))
    amax = blocks.abs().amax(-1)
    if fmt == "mxfp4":
        x = (torch.floor(torch.log2(amax.clamp_min(2.0 ** -126))) - 2).clamp(-127, 127)
        scales = (x + 127).to(torch.uint8)
        inv = torch.exp2(-x)
        g = torch.ones(w.shape[:-2], dtype=torch.float32, device=w.device)
    else:
        g = 448.0 * 6.0 / amax.amax((-1, -2))
        s = (amax * g[..., None, None] / 6.0).clamp_max(448.0).to(torch.float8_e4m3fn)
        scales = s.view(torch.uint8)
        inv = g[..., None, None] / s.float().clamp_min(2.0 ** -9)
    v = blocks * inv[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scales.contiguous(), g


def _fp4_weights(gen, shape, fmt):
    """Normal weights of the usual size, quantized a matrix at a time."""
    lead, (n, kk) = shape[:-2], shape[-2:]
    parts = [_quantize(_normal(gen, (n, kk), kk ** -0.5, torch.float32), fmt) for _ in range(math.prod(lead))]
    codes, scales, g = (torch.stack(p).reshape(lead + p[0].shape) for p in zip(*parts))
    return codes, scales, g


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _normal(gen, (T, H))
        # a residual stream: rows of different size
        s["residual"] = (_normal(gen, (T, H), 2.0, torch.float32)
                         * torch.exp(_normal(gen, (T, 1), 0.5, torch.float32))).to(torch.bfloat16)
        s["weight"] = (1.0 + _normal(gen, (H,), 0.1, torch.float32)).to(torch.bfloat16)
        s["eps"] = 1e-6
        s["residual_out"] = torch.empty_like(s["x"])
        return s
    if case["op"] == "gemv":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = _normal(gen, (T, K))
        s["codes"], s["scales"], g = _fp4_weights(gen, (N, K), case["fmt"])
        s["g"] = float(g)
        return s
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    s["x"] = _normal(gen, (T, H))
    s["logits"] = _normal(gen, (T, E), 1.0, torch.float32)
    if case["fmt"] == "bf16":
        s["w13"] = _normal(gen, (E, 2 * I, H), H ** -0.5)
        s["w2"] = _normal(gen, (E, H, I), I ** -0.5)
    else:
        s["w13"], s["w13_scales"], s["w13_g"] = _fp4_weights(gen, (E, 2 * I, H), case["fmt"])
        s["w2"], s["w2_scales"], s["w2_g"] = _fp4_weights(gen, (E, H, I), case["fmt"])
    # the buffers that a decode loop keeps
    s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    s["topk_ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
    s["topk_weights"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    s["workspace"] = None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _dequant(codes, scales, g, fmt):
    """Codes [..., n/2] and scales [..., n/block] -> float32 [..., n]."""
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = values[nib.int()].unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "mxfp4":
        sv = torch.exp2(scales.float() - 127.0)
    else:
        sv = scales.view(torch.float8_e4m3fn).float()
        sv = sv / (g[..., None, None] if isinstance(g, torch.Tensor) else g)
    return (v * sv[..., None]).flatten(-2)


def _mxfp8(y):
    """bfloat16 [T, n] -> E4M3 values and E8M0 scale values."""
    b = y.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 1   # floor(log2 amax)
    x = torch.where(amax > 0, e - 8, -127).clamp(-127, 127)
    codes = (b * torch.exp2(-x.float())[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (x + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _norm_plain(s):
    h = s["x"].float() + s["residual"].float()
    y = (s["weight"].float() * (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]))).to(torch.bfloat16)
    r = h.to(torch.bfloat16)
    if s["out"] == "bf16":
        return {"y": y, "residual": r}
    codes, scales = _mxfp8(y)
    res = {"codes": codes, "scales": scales, "residual": r}
    return res if s["out"] == "mxfp8" else {"y": y, **res}


def _norm_own(s):
    import memory_bound_moe_gb300 as moe
    if s["out"] == "bf16":
        y, r = moe.moe_add_rmsnorm(s["x"], s["residual"], s["weight"], 0.0, s["eps"],
                                   residual_out=s["residual_out"])
        return {"y": y, "residual": r}
    y = torch.empty_like(s["x"]) if s["out"] == "both" else None
    codes, scales, r = moe.moe_add_rmsnorm_mxfp8(s["x"], s["residual"], s["weight"], 0.0, s["eps"], out=y,
                                                 residual_out=s["residual_out"])
    res = {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu), "residual": r}
    return res if y is None else {"y": y, **res}


def _gemv_plain(s):
    w = _dequant(s["codes"], s["scales"], s["g"], s["fmt"])
    return (s["x"].float() @ w.t()).to(torch.bfloat16 if s["out"] == "bf16" else torch.float32)


def _gemv_own(s):
    import memory_bound_moe_gb300 as moe
    return moe.moe_gemv_fp4(s["x"], s["codes"], s["scales"], s["fmt"], s["g"],
                            out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)


def _layer_plain(s):
    k, E, I = s["k"], s["E"], s["I"]
    x = s["x"].float()
    T = x.shape[0]
    p = torch.exp(s["logits"] - s["logits"].amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    # ties go to the lower expert
    ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)

    few = T * k < E   # either the chosen experts' weights, slot by slot, or all experts

    def weights(name):
        pick = (lambda t: t[ids.flatten()]) if few else (lambda t: t)
        if s["fmt"] == "bf16":
            return pick(s[name]).float()
        return _dequant(pick(s[name]), pick(s[name + "_scales"]), pick(s[name + "_g"]), s["fmt"])

    xs = x[:, None].expand(-1, k, -1).reshape(T * k, 1, -1) if few else x.expand(E, -1, -1)
    gu = xs @ weights("w13").transpose(1, 2)             # [S, 1, 2I] or [E, T, 2I]
    a = gu[..., :I] / (1.0 + torch.exp(-gu[..., :I])) * gu[..., I:]
    y = a @ weights("w2").transpose(1, 2)
    y = y.view(T, k, -1) if few else y[ids, torch.arange(T, device=x.device)[:, None]]
    out = (w[..., None] * y).sum(1)
    return {"out": out.to(torch.bfloat16), "topk_ids": ids.int(), "topk_weights": w}


def _layer_own(s):
    import memory_bound_moe_gb300 as moe
    if s["workspace"] is None:
        s["workspace"] = torch.empty(moe.moe_layer_workspace_size(s["T"], s["E"], s["k"], s["H"], s["I"]),
                                     dtype=torch.uint8, device=DEV)
    bufs = dict(out=s["out"], topk_ids=s["topk_ids"],
                topk_weights=s["topk_weights"], workspace=s["workspace"])
    if s["fmt"] == "bf16":
        out = moe.moe_layer(s["logits"], s["x"], s["w13"], s["w2"], s["k"], s["renorm"], **bufs)
    else:
        g13, g2 = (s["w13_g"], s["w2_g"]) if s["fmt"] == "nvfp4" else (None, None)
        out = moe.moe_layer_fp4(s["logits"], s["x"], s["w13"], s["w13_scales"], s["w2"], s["w2_scales"], s["k"],
                                s["renorm"], s["fmt"], g13, g2, **bufs)
    return {"out": out, "topk_ids": s["topk_ids"], "topk_weights": s["topk_weights"]}


def run(s):
    if own:
        return {"norm": _norm_own, "gemv": _gemv_own, "layer": _layer_own}[s["op"]](s)
    return {"norm": _norm_plain, "gemv": _gemv_plain, "layer": _layer_plain}[s["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------

def _weights64(codes, scales, g, fmt):
    """One matrix's values: a table look-up per code, times its block's scale."""
    mag = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    lo, hi = (codes & 0x0F).long(), (codes >> 4).long()
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    v[:, 0::2] = mag[lo & 7] * (1 - 2 * (lo >> 3))
    v[:, 1::2] = mag[hi & 7] * (1 - 2 * (hi >> 3))
    if fmt == "mxfp4":
        s = torch.pow(2.0, scales.double() - 127)
    else:
        b = scales.long()   # E4M3 from its fields
        e, m = (b >> 3) & 15, (b & 7).double()
        s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, e.double() - 7)) / float(g)
    return v * s.repeat_interleave(BLOCK[fmt], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + s["residual"].double()
        y = s["weight"].double() * h / torch.sqrt(torch.sum(h ** 2, 1, keepdim=True) / case["H"] + s["eps"])
        res = {"residual": h}
        if case["out"] != "mxfp8":
            res["y"] = y
        if case["out"] != "bf16":
            # the codes are defined on the bfloat16 values of y
            b = y.to(torch.bfloat16).double().view(case["T"], -1, 32)
            x = torch.floor(torch.log2(b.abs().amax(2))) - 8
            x = x.masked_fill(b.abs().amax(2) == 0, -127).clamp(-127, 127)
            v = b / torch.pow(2.0, x)[..., None]
            # nearest multiple of the E4M3 step at v's binade, ties to even
            step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            res["codes"] = (torch.round(v / step) * step).clamp(-448, 448).view(case["T"], -1)
            res["scales"] = torch.pow(2.0, x)
        return res
    if case["op"] == "gemv":
        return s["x"].double() @ _weights64(s["codes"], s["scales"], s["g"], case["fmt"]).T
    T, H, E, k, I = (case[n] for n in ("T", "H", "E", "k", "I"))
    l = s["logits"].double()
    p = torch.softmax(l, 1)
    ids = [sorted(range(E), key=lambda e, r=r: (-r[e], e))[:k] for r in l.tolist()]
    w = torch.stack([p[t, ids[t]] for t in range(T)])
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in sorted({e for r in ids for e in r}):
        ts = [t for t in range(T) if e in ids[t]]
        if case["fmt"] == "bf16":
            w13, w2 = s["w13"][e].double(), s["w2"][e].double()
        else:
            w13 = _weights64(s["w13"][e], s["w13_scales"][e], s["w13_g"][e], case["fmt"])
            w2 = _weights64(s["w2"][e], s["w2_scales"][e], s["w2_g"][e], case["fmt"])
        xt = s["x"][ts].double()
        gate, up = xt @ w13[:I].T, xt @ w13[I:].T
        a = gate * torch.sigmoid(gate) * up
        we = torch.stack([w[t, ids[t].index(e)] for t in ts])
        out[ts] += we[:, None] * (a @ w2.T)
    return {"out": out, "topk_ids": None, "topk_weights": w}
