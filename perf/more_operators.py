"""Cases that measure a decode step's cache: attention of one new token per
sequence over a paged key-value cache, the step's block tables and slot maps,
and the rotary embedding with the write of keys and values into the cache.

Each operator also stands here in its plain form (elementary torch operations
in float32, whole numbers in int64), which runs without the library; with
``own`` set, ``run`` makes the library's calls instead. ``exact`` evaluates
the definitions in float64.
"""
import math

import torch

own = False

DEV = "cuda"
SCALES = {"bf16": (1.0, 1.0), "e4m3": (1 / 64, 3 / 256)}   # of keys and values in the cache
BYTES = {"bf16": 2, "e4m3": 1}
MAX_BYTES = 1.09e9   # of keys and values read by one attention, the largest listed


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    """Heads are those of the library's QK norm tests (32 over 4, 64 over 8 and
    8 over 8 heads, 16 over 2 of 256); batches and prompts those of its decode,
    skewed and prefill workloads (16, 1023 and 8192 tokens)."""
    return [
        # one user's token after a short conversation: latency
        dict(name="attention one user", op="attention", B=1, Hq=32, Hkv=4, D=128, lo=1023, hi=1023, page=16,
             cache="bf16", window=0, layout="token"),
        # a decode batch of very different lengths
        dict(name="attention decode", op="attention", B=16, Hq=64, Hkv=8, D=128, lo=1, hi=8192, page=64,
             cache="bf16", window=0, layout="token"),
        # two long documents: few rows, so the length has to be split
        dict(name="attention long", op="attention", B=2, Hq=64, Hkv=8, D=128, lo=130001, hi=131072, page=64,
             cache="bf16", window=0, layout="token"),
        # the fullest batch, pages of 16: the largest, with the two beside it
        dict(name="attention full batch", op="attention", B=256, Hq=32, Hkv=4, D=128, lo=17, hi=4096, page=16,
             cache="bf16", window=0, layout="token"),
        # an 8-bit cache, stored head by head inside a page
        dict(name="attention e4m3", op="attention", B=64, Hq=64, Hkv=8, D=128, lo=1, hi=16384, page=32,
             cache="e4m3", window=0, layout="head"),
        # a query head per key head of 64, pages of one token, an odd batch with an empty sequence
        dict(name="attention heads of 64", op="attention", B=33, Hq=8, Hkv=8, D=64, lo=0, hi=5000, page=1,
             cache="bf16", window=0, layout="token"),
        # heads of 256 that look back over a window only
        dict(name="attention window", op="attention", B=24, Hq=16, Hkv=2, D=256, lo=500, hi=32768, page=16,
             cache="bf16", window=1023, layout="token"),
        # the new tokens of a decode batch: latency
        dict(name="append decode", op="append", N=16, Hq=64, Hkv=8, D=128, rot=128, pairs=False, page=64,
             cache="bf16", pad=0),
        # a prompt chunk, q, k and v sliced from one projection's rows: bandwidth
        dict(name="append prefill", op="append", N=8192, Hq=32, Hkv=4, D=128, rot=128, pairs=False, page=16,
             cache="bf16", pad=0),
        # an odd chunk with padding behind it, rotated in part and in pairs, into an 8-bit cache
        dict(name="append e4m3", op="append", N=1023, Hq=16, Hkv=2, D=256, rot=64, pairs=True, page=32,
             cache="e4m3", pad=57),
        # one more token for every request of a decode batch
        dict(name="table decode", op="table", B=16, page=64, most=1, N=16, longest=8192),
        # a large batch in which some requests bring a chunk of their prompt
        dict(name="table mixed", op="table", B=1023, page=16, most=256, N=32768, longest=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "table"])
    while True:
        if op == "attention":
            Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
            c = dict(op=op, B=_log(rng, 1, 256), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 256]), lo=0,
                     hi=_log(rng, 1, 131072), page=2 ** rng.randint(0, 8), cache=rng.choice(["bf16", "e4m3"]),
                     window=0 if rng.random() < 0.7 else _log(rng, 1, 4096), layout=rng.choice(["token", "head"]))
            c["lo"] = rng.randint(0, c["hi"])
            # the plain form holds the padded batch in float32; it costs no more than a listed one's
            if c["B"] * c["hi"] * Hkv * c["D"] * 4 <= 2 * MAX_BYTES and c["B"] * c["hi"] * c["Hq"] <= 2 ** 27:
                return c
        elif op == "append":
            Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
            c = dict(op=op, N=_log(rng, 1, 8192), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 256]),
                     pairs=rng.random() < 0.5, page=2 ** rng.randint(0, 8), cache=rng.choice(["bf16", "e4m3"]),
                     pad=rng.choice([0, 0, rng.randint(1, 100)]))
            c["rot"] = c["D"] if rng.random() < 0.5 else rng.choice([0, 16, 32, 64])
            if c["N"] * (c["Hq"] + 2 * Hkv) * c["D"] <= 8192 * 40 * 128:
                return c
        else:
            c = dict(op=op, B=_log(rng, 1, 4096), page=2 ** rng.randint(0, 8), most=_log(rng, 1, 2048),
                     N=_log(rng, 1, 32768), longest=_log(rng, 1, 32768), scarce=rng.random() < 0.3)
            if c["B"] * -(-(c["longest"] + c["most"]) // c["page"]) <= 2 ** 24:
                return c


def _lengths(c):
    """The sequences' lengths, evenly spread from lo to hi (their order is the seed's)."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def work(c):
    if c["op"] == "attention":
        read = [min(n, c["window"] or n) for n in _lengths(c)]
        pages = sum(-(-n // c["page"]) for n in read)
        return {"bytes": 2 * sum(read) * c["Hkv"] * c["D"] * BYTES[c["cache"]] + 4 * c["B"] * c["Hq"] * (c["D"] + 1)
                + 4 * pages + 4 * c["B"],
                "flops": 4 * sum(read) * c["Hq"] * c["D"]}
    if c["op"] == "append":
        N, D = c["N"], c["D"]
        return {"bytes": N * (4 * c["Hq"] * D + 2 * c["Hkv"] * D * (2 + BYTES[c["cache"]]) + 4 * c["rot"] + 12),
                "flops": 6 * N * (c["Hq"] + c["Hkv"]) * c["rot"] / 2}
    new = min(c["N"], c["B"] * c["most"]) / c["page"]   # pages, about
    return {"bytes": 16 * c["B"] + 12 * c["N"] + 8 * new + 4 * c["B"], "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=gen)


def _cache(gen, pages, c):
    """Keys or values of unit size, [pages, page, Hkv, D]; stored token by
    token, or head by head and seen through a transposed view."""
    def values(scale):
        shape = (pages, c["page"], c["Hkv"], c["D"])
        if c.get("layout") == "head":
            shape = (pages, c["Hkv"], c["page"], c["D"])
        if c["cache"] == "bf16":
            t = _normal(gen, shape)
        else:
            t = _normal(gen, shape, 1 / scale).clamp_(-448, 448).to(torch.float8_e4m3fn)
        return t.transpose(1, 2) if c.get("layout") == "head" else t
    return tuple(values(s) for s in SCALES[c["cache"]])


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    c = case
    s["k_scale"], s["v_scale"] = SCALES.get(c.get("cache"), (1.0, 1.0))
    perm = lambda n: torch.randperm(n, generator=gen, device=DEV)   # noqa: E731
    if c["op"] == "attention":
        B, P = c["B"], c["page"]
        s["lengths"] = _int(_lengths(c))[perm(B)].contiguous()
        s["max_pages"] = M = max(1, -(-c["hi"] // P))
        used = sum(-(-n // P) for n in _lengths(c))
        s["pages"] = pages = used + 1
        s["k_cache"], s["v_cache"] = _cache(gen, pages, c)
        # pages were handed out as they came free: in no order
        have = (s["lengths"].long() + P - 1) // P
        at = torch.arange(M, device=DEV)[None]
        row = (have.cumsum(0) - have)[:, None] + at
        s["block_table"] = torch.where(at < have[:, None], perm(pages)[row.clamp_max(pages - 1)], 0).int()
        # scores of a few units: neither flat nor one token's alone
        s["q"] = _normal(gen, (B, c["Hq"], c["D"]), 2.0)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, c["Hq"]), dtype=torch.float32, device=DEV)
        s["handle"] = s["workspace"] = None
    elif c["op"] == "append":
        N, Hq, Hkv, D, P = (c[n] for n in ("N", "Hq", "Hkv", "D", "page"))
        rows = N + c["pad"]
        # the output rows of one projection: q, k and v beside each other
        qkv = _normal(gen, (rows, (Hq + 2 * Hkv) * D), 1.5)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
        pages = -(-N // P) * 2
        s["k_cache"], s["v_cache"] = _cache(gen, pages, c)
        slots = perm(pages)[torch.arange(N, device=DEV) // P] * P + torch.arange(N, device=DEV) % P
        s["slots"] = torch.cat([slots, slots.new_full((c["pad"],), -1)])
        positions = torch.randint(0, 20000, (1,), generator=gen, device=DEV) + torch.arange(N, device=DEV) % 5000
        s["positions"] = torch.cat([positions, positions.new_zeros(c["pad"])]).int()
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / max(1, c["rot"]))
        angle = torch.arange(25001, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.zeros((rows, Hq, D), dtype=torch.bfloat16, device=DEV)
        s["handle"] = None
    else:
        B, P, N = c["B"], c["page"], c["N"]
        s["max_pages"] = M = -(-(c["longest"] + c["most"]) // P)
        rand = lambda hi: torch.randint(0, hi + 1, (B,), generator=gen, device=DEV)   # noqa: E731
        s["cached"] = rand(c["longest"]).int()
        # most requests bring one token, a few a chunk; a step that has more than N in all turns some away
        chunk = (rand(31) == 0).long() * rand(c["most"])
        s["added"] = torch.maximum(torch.ones_like(chunk), chunk).int() if B > 1 else _int([c["most"]])
        have = (s["cached"].long() + P - 1) // P
        pages = int(have.sum())
        ids = perm(pages + B + N // P + 1)
        at = torch.arange(M, device=DEV)[None]
        row = (have.cumsum(0) - have)[:, None] + at
        s["block_table"] = torch.where(at < have[:, None], ids[row.clamp_max(len(ids) - 1)], -1).int()
        # enough for all, or so few that the last requests have to wait
        s["free_pages"] = ids[pages:pages + 1 + B // 3 if c.get("scarce") else None].int().contiguous()
        s["free_count"] = _int([len(s["free_pages"])])
        i32 = dict(dtype=torch.int32, device=DEV)
        # the buffers that a captured decode step writes
        s["out"] = (torch.empty(B, **i32), torch.empty(B + 1, **i32), torch.empty(N, **i32),
                    torch.empty(N, dtype=torch.int64, device=DEV), torch.empty(1, **i32), torch.empty(1, **i32))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _attention_plain(s):
    B, Hkv, D, P, M = (s[n] for n in ("B", "Hkv", "D", "page", "max_pages"))
    G = s["Hq"] // Hkv
    table = s["block_table"].long()
    k, v = (s[n][table].float().flatten(1, 2) for n in ("k_cache", "v_cache"))         # [B, M P, Hkv, D]
    q = s["q"].float().view(B, Hkv, G, D) * (s["k_scale"] / math.sqrt(D))
    score = q @ k.permute(0, 2, 3, 1)                                                   # [B, Hkv, G, M P]
    n = s["lengths"].long()[:, None]
    at = torch.arange(M * P, device=n.device)[None]
    seen = (at < n) & (at >= (n - s["window"] if s["window"] else 0 * n))
    score = torch.where(seen[:, None, None], score, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = (p @ v.transpose(1, 2)) * (s["v_scale"] / torch.where(total == 0, 1.0, total))
    lse = (m + torch.log(total)).view(B, -1)
    return {"out": out.view(B, -1, D).to(torch.bfloat16), "lse": lse}


def _handle(s):
    import memory_bound_moe_gb300 as moe
    if s["handle"] is None:
        s["handle"] = moe.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return s["handle"]


def _attention_own(s):
    import memory_bound_moe_gb300 as moe
    cache = _handle(s)
    if s["workspace"] is None:
        s["workspace"] = torch.empty(moe.moe_paged_attention_workspace_size(s["B"], s["Hq"], s["Hkv"], s["D"]),
                                     dtype=torch.uint8, device=DEV)
    out = moe.moe_paged_attention(s["q"], cache, s["block_table"], s["lengths"], window=s["window"], out=s["out"],
                                  lse=s["lse"], workspace=s["workspace"])
    return {"out": out, "lse": s["lse"]}


def _rotate(x, cos, sin, rot, pairs):
    """x [rows, heads, D] with its first rot columns rotated; cos, sin [rows, rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _append_plain(s):
    keep = (s["slots"] >= 0).nonzero().flatten()
    slots = s["slots"][keep]
    cos, sin = s["cos_sin"][s["positions"][keep].long()].chunk(2, 1)
    q, k = (_rotate(s[n][keep].float(), cos, sin, s["rot"], s["pairs"]) for n in ("q", "k"))
    s["q_out"][keep] = q.to(torch.bfloat16)
    at = (slots // s["page"], slots % s["page"])
    if s["cache"] == "bf16":
        s["k_cache"][at] = k.to(torch.bfloat16)
        s["v_cache"][at] = s["v"][keep]
    else:
        code = lambda x, scale: (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)   # noqa: E731
        s["k_cache"].view(torch.uint8)[at] = code(k, s["k_scale"])
        s["v_cache"].view(torch.uint8)[at] = code(s["v"][keep].float(), s["v_scale"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _append_own(s):
    import memory_bound_moe_gb300 as moe
    moe.moe_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], _handle(s),
                      interleaved=s["pairs"], q_out=s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _table_plain(s):
    P, N, M = s["page"], s["N"], s["max_pages"]
    c, a = s["cached"].long(), s["added"].long()
    end = a.cumsum(0)
    have, need = (c + P - 1) // P, (c + a + P - 1) // P
    fits = (need <= M) & (end <= N)
    new = torch.where(fits, need - have, 0)
    taken = new.cumsum(0)
    free = s["free_count"].long()
    ok = fits & ((new == 0) | (taken <= free))
    # the new pages of request b: entries have .. need - 1 of its row, off the stack's top in order
    at = torch.arange(M, device=c.device)[None]
    fresh = ok[:, None] & (at >= have[:, None]) & (at < need[:, None])
    index = free - 1 - (taken - new)[:, None] - (at - have[:, None])
    table = torch.where(fresh, s["free_pages"][index.clamp(0, len(s["free_pages"]) - 1)], s["block_table"])
    s["block_table"].copy_(table)
    i = torch.arange(N, device=c.device)
    b = torch.searchsorted(end, i, right=True).clamp_max(len(c) - 1)
    there = (i < end[-1]) & ok[b]
    pos = torch.where(there, c[b] + i - (end - a)[b], 0)
    slots = torch.where(there, table[b, pos // P].long() * P + pos % P, -1)
    return {"block_table": s["block_table"], "lengths": torch.where(ok, c + a, c).int(),
            "starts": torch.cat([end - a, end[-1:]]).int(), "positions": pos.int(), "slots": slots,
            "free_count": free.int() - torch.where(taken <= free, taken, 0).amax().int(),
            "refused": (~ok).sum().int().view(1)}


def _table_own(s):
    import memory_bound_moe_gb300 as moe
    t = moe.moe_page_table(s["cached"], s["added"], s["block_table"], s["free_pages"], s["free_count"], s["page"],
                           s["N"], out=moe.PageTable(*s["out"]))
    return {"block_table": s["block_table"], **t._asdict()}


def run(s):
    if own:
        return {"attention": _attention_own, "append": _append_own, "table": _table_own}[s["op"]](s)
    return {"attention": _attention_plain, "append": _append_plain, "table": _table_plain}[s["op"]](s)


# ---------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "table":
        return None   # whole numbers alone
    if c["op"] == "attention":
        B, Hq, D, P = c["B"], c["Hq"], c["D"], c["page"]
        G = Hq // c["Hkv"]
        out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lengths"].tolist()):
            first = max(0, n - c["window"]) if c["window"] else 0
            if n == first:
                continue
            j = torch.arange(first, n, device=DEV)
            page, row = s["block_table"][b].long()[j // P], j % P
            k, v = (s[name][page, row].double() for name in ("k_cache", "v_cache"))   # [n, Hkv, D]
            for h in range(c["Hkv"]):
                heads = slice(h * G, (h + 1) * G)
                x = s["q"][b, heads].double() @ k[:, h].T * s["k_scale"] / D ** 0.5
                lse[b, heads] = torch.logsumexp(x, 1)
                out[b, heads] = torch.softmax(x, 1) @ v[:, h] * s["v_scale"]
        return {"out": out, "lse": lse}
    N, rot = c["N"], c["rot"]
    cs = s["cos_sin"].double()[s["positions"][:N].long()]
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
    res = {}
    for name in ("q", "k"):
        x = s[name][:N].double()
        y = x.clone()
        if c["pairs"]:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        res[name] = y
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    q[:N] = res["q"]
    page, row = s["slots"][:N] // c["page"], s["slots"][:N] % c["page"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[page, row] = (res["k"] / s["k_scale"]).clamp(-448, 448) if c["cache"] == "e4m3" else res["k"]
    vc[page, row] = (s["v"][:N].double() / s["v_scale"]).clamp(-448, 448) if c["cache"] == "e4m3" else s["v"][:N].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}
