"""moe_layer and moe_layer_fp4 on the GPU against the definition in float64
(bounds: few_reference.py); the routing against moe_route, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from few_reference import check_layer, random_fp4, weights64

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_moe_gb300 import build
    build.build()
    return torch.device("cuda:0")


class Layer:
    def __init__(self, E, H, I, fmt, dev, seed):
        self.E, self.H, self.I, self.fmt = E, H, I, fmt
        rng = np.random.default_rng(seed)
        if fmt == "bf16":
            bf = lambda shape, n: torch.from_numpy((rng.standard_normal(shape) / n ** 0.5).astype(np.float32)).to(torch.bfloat16)
            self.w13, self.w2 = bf((E, 2 * I, H), H).to(dev), bf((E, H, I), I).to(dev)
            self.values = lambda e: (self.w13[e].double().cpu().numpy(), self.w2[e].double().cpu().numpy())
            return
        self.h13, self.h2 = random_fp4(rng, (E, 2 * I, H), fmt), random_fp4(rng, (E, H, I), fmt)
        if fmt == "nvfp4":   # products of ordinary size: about 1 / sqrt(k) after the tensor scale
            self.g = [(rng.uniform(50, 200, E) * n ** 0.5).astype(np.float32) for n in (H, I)]
        else:
            self.g = [np.ones(E, np.float32)] * 2
        up = lambda a: torch.from_numpy(a).to(dev)
        self.d = [up(self.h13[0]), up(self.h13[1]), up(self.h2[0]), up(self.h2[1])]
        self.gd = [up(g) for g in self.g] if fmt == "nvfp4" else [None, None]
        self.values = lambda e: (weights64(self.h13[0][e], self.h13[1][e], fmt, self.g[0][e]),
                                 weights64(self.h2[0][e], self.h2[1][e], fmt, self.g[1][e]))

    def __call__(self, logits, x, k, renorm, **kw):
        from memory_bound_moe_gb300 import moe_layer, moe_layer_fp4
        if self.fmt == "bf16":
            return moe_layer(logits, x, self.w13, self.w2, k, renorm, **kw)
        return moe_layer_fp4(logits, x, *self.d, k, renorm, self.fmt, *self.gd, **kw)


def tokens(T, E, H, dev, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, E, generator=g).to(dev), torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev)


def run_and_check(layer, logits, x, k, renorm, what):
    from memory_bound_moe_gb300 import moe_route
    T, dev = logits.shape[0], logits.device
    ids = torch.full((T, k), -5, dtype=torch.int32, device=dev)
    wts = torch.full((T, k), float("nan"), dtype=torch.float32, device=dev)
    out = layer(logits, x, k, renorm, topk_ids=ids, topk_weights=wts)
    r = moe_route(logits, k, renorm)
    assert torch.equal(ids, r.topk_ids) and torch.equal(wts, r.topk_weights), what
    check_layer(out, ids.cpu().numpy(), wts.double().cpu().numpy(), x, layer.values, layer.H, layer.I, what)
    assert torch.equal(out, layer(logits, x, k, renorm)), what       # the same bits, without the routing outputs
    return out


# T, E, k, H, I
SHAPES = [(1, 1, 1, 32, 32), (1, 8, 2, 64, 96), (2, 3, 3, 160, 32), (7, 16, 4, 288, 160), (8, 64, 8, 256, 128),
          (9, 17, 2, 96, 352), (16, 128, 8, 512, 96), (17, 33, 5, 64, 64), (31, 8, 2, 320, 192), (32, 256, 8, 128, 64),
          (32, 8, 2, 512, 448), (32, 1024, 16, 64, 32), (5, 600, 16, 96, 64), (32, 2, 2, 2880, 160), (3, 4, 1, 160, 2880)]


@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("renorm", [True, False])
def test_against_float64(dev, T, E, k, H, I, fmt, renorm):
    layer = Layer(E, H, I, fmt, dev, T + E + H + I)
    logits, x = tokens(T, E, H, dev, T * E + k)
    run_and_check(layer, logits, x, k, renorm, f"T={T} E={E} k={k} H={H} I={I} {fmt}")


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 8, 8), (3, 5, 2, 24, 40), (13, 9, 3, 200, 72), (32, 6, 2, 1000, 424)])
def test_bf16_rows_of_16_bytes(dev, T, E, k, H, I):
    layer = Layer(E, H, I, "bf16", dev, H)
    logits, x = tokens(T, E, H, dev, I)
    run_and_check(layer, logits, x, k, True, f"H={H} I={I}")


@pytest.mark.parametrize("fmt", FMTS)
def test_all_tokens_on_one_expert_and_ties(dev, fmt):
    layer = Layer(8, 96, 64, fmt, dev, 1)
    logits, x = tokens(32, 8, 96, dev, 2)
    logits[:, 5] = 50.0
    run_and_check(layer, logits, x, 1, True, "one expert")
    logits.zero_()                                                   # ties: experts 0 and 1
    run_and_check(layer, logits, x, 2, False, "ties")


@pytest.mark.parametrize("fmt", FMTS)
def test_equals_the_call_by_call_path(dev, fmt):
    """A decode step as it would be used: norm with the residual, router
    logits, the layer; the layer's result against route, expand, products,
    SwiGLU and combine with the same weights."""
    from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_combine, moe_expand, moe_route, moe_swiglu
    T, E, k, H, I = 12, 16, 4, 256, 160
    layer = Layer(E, H, I, fmt, dev, 9)
    _, x = tokens(T, E, H, dev, 3)
    residual = torch.randn(T, H, device=dev).to(torch.bfloat16)
    y, residual = moe_add_rmsnorm(x, residual, torch.ones(H, dtype=torch.bfloat16, device=dev))
    router = torch.randn(E, H, device=dev) / 16
    logits = y.float() @ router.t()
    out = run_and_check(layer, logits, y, k, True, "decode step")
    r = moe_route(logits, k, True)
    xe = moe_expand(y, r.inv_perm, k).float()
    counts = r.expert_counts.tolist()
    gu, eo = [], []
    for e, rows in enumerate(torch.split(xe, counts)):
        gu.append(rows @ torch.from_numpy(layer.values(e)[0]).to(dev).float().t())
    act = moe_swiglu(torch.cat(gu).to(torch.bfloat16).contiguous()).float()
    for e, rows in enumerate(torch.split(act, counts)):
        eo.append(rows @ torch.from_numpy(layer.values(e)[1]).to(dev).float().t())
    ref = moe_combine(torch.cat(eo).to(torch.bfloat16).contiguous(), r.topk_weights, r.inv_perm)
    # that path rounds gate_up, act, expert_out and out to bfloat16 and the
    # layer a and out; errors of 2^-8 / sqrt(3) of the norm each, gate_up's
    # entering twice (gate and up): under 3 * 2^-8 together
    rel = float((out.double() - ref.double()).norm() / ref.double().norm())
    assert rel <= 3 * 2.0 ** -8, rel


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 6, 19])
def test_decode_step_in_a_graph(dev, fmt, T):
    """Norm with the residual, 4-bit router and layer, as one captured step
    that is replayed on new tokens: each call against its definition."""
    from few_reference import check_gemv
    from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_gemv_fp4, moe_layer_workspace_size
    E, k, H, I = 24, 4, 288, 160
    layer = Layer(E, H, I, fmt, dev, 20)
    rc, rs = random_fp4(np.random.default_rng(21), (E, H), fmt)
    rg = 300.0 if fmt == "nvfp4" else 1.0
    rcd, rsd = torch.from_numpy(rc).to(dev), torch.from_numpy(rs).to(dev)
    weight = torch.ones(H, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(moe_layer_workspace_size(T, E, k, H, I), dtype=torch.uint8, device=dev)
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    residual = torch.zeros_like(x)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    wts = torch.empty((T, k), dtype=torch.float32, device=dev)

    def step():
        y, _ = moe_add_rmsnorm(x, residual, weight)
        logits = moe_gemv_fp4(y, rcd, rsd, fmt, rg, out_dtype=torch.float32)
        return y, logits, layer(logits, y, k, True, topk_ids=ids, topk_weights=wts, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, logits, out = step()
    for rep in range(3):
        x.copy_(torch.randn((T, H), generator=torch.Generator().manual_seed(rep)).to(torch.bfloat16))
        sum_ = residual.double().cpu() + x.double().cpu()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(residual.cpu(), sum_.float().to(torch.bfloat16))
        ref = sum_ / torch.sqrt((sum_ ** 2).mean(1, keepdim=True) + 1e-6)
        # half a step of bfloat16, and the float32 sum, root and products: 2^-16
        assert ((y.double().cpu() - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -134).all()
        check_gemv(logits, y, weights64(rc, rs, fmt, rg), "router")
        check_layer(out, ids.cpu().numpy(), wts.double().cpu().numpy(), y, layer.values, H, I, "layer")


@pytest.mark.parametrize("fmt", FMTS)
def test_unchosen_weights_do_not_matter_and_tokens_stay_apart(dev, fmt):
    E, H, I, T, k = 12, 64, 64, 10, 2
    layer = Layer(E, H, I, fmt, dev, 4)
    logits, x = tokens(T, E, H, dev, 5)
    logits[:, [3, 7, 11]] = -100.0
    out = layer(logits, x, k, True)
    for e in (3, 7, 11):
        if fmt == "bf16":
            layer.w13[e] = float("nan")
            layer.w2[e] = float("nan")
        else:
            bad = 255 if fmt == "mxfp4" else 127
            layer.d[1][e] = bad
            layer.d[3][e] = bad
    x2 = x.clone()
    x2[4] = float("nan")
    got = layer(logits, x2, k, True)
    assert got[4].isnan().all()
    keep = [t for t in range(T) if t != 4]
    assert torch.equal(got[keep], out[keep])


@pytest.mark.parametrize("fmt", FMTS)
def test_buffers_streams_and_graphs(dev, fmt):
    from memory_bound_moe_gb300 import moe_layer_workspace_size
    E, H, I, T, k = 16, 128, 96, 6, 4
    layer = Layer(E, H, I, fmt, dev, 6)
    logits, x = tokens(T, E, H, dev, 7)
    want = layer(logits, x, k, True)
    need = moe_layer_workspace_size(T, E, k, H, I)
    ws = torch.full((need + 256,), 171, dtype=torch.uint8, device=dev)
    buf = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device=dev)
    layer(logits, x, k, True, out=buf[:T], workspace=ws[:need])
    assert torch.equal(buf[:T], want) and (buf[T:] == 7).all() and (ws[need:] == 171).all()
    # two graphs that captured the same workspace, replayed in order, with new inputs
    outs, graphs, ins = [], [], []
    for i in range(2):
        li, xi = logits.clone(), x.clone()
        o = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(li, xi, k, True, out=o, workspace=ws[:need])
        outs.append(o)
        graphs.append(graph)
        ins.append((li, xi))
    for rep in range(3):
        for i in range(2):
            li, xi = tokens(T, E, H, dev, 100 + 10 * rep + i)
            ins[i][0].copy_(li)
            ins[i][1].copy_(xi)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], layer(*ins[i], k, True))
    # calls on two streams at once, each with a workspace of its own
    streams = [torch.cuda.Stream() for _ in range(2)]
    batches = [tokens(T, E, H, dev, 200 + i) for i in range(2)]
    refs = [layer(*b, k, True) for b in batches]
    torch.cuda.synchronize()
    got = [[layer(*b, k, True, stream=s) for _ in range(8)] for b, s in zip(batches, streams)]
    torch.cuda.synchronize()
    for r, gs in zip(refs, got):
        assert all(torch.equal(r, g) for g in gs)


@pytest.mark.parametrize("fmt", FMTS)
def test_operands_at_16_bytes(dev, fmt):
    """x and the weights 16, but not 32 bytes behind a boundary: the same bits."""
    def moved(t):
        b = t.contiguous().view(torch.uint8).flatten()
        buf = torch.empty(b.numel() + 64, dtype=torch.uint8, device=dev)
        assert buf.data_ptr() % 32 == 0
        return buf[16:16 + b.numel()].copy_(b).view(t.dtype).view(t.shape)

    for T in (3, 20):
        layer = Layer(6, 608, 320, fmt, dev, 14)
        logits, x = tokens(T, 6, 608, dev, 15)
        want = run_and_check(layer, logits, x, 2, True, "aligned")
        if fmt == "bf16":
            layer.w13, layer.w2 = moved(layer.w13), moved(layer.w2)
        else:
            layer.d = [moved(t) for t in layer.d]
        assert torch.equal(want, layer(logits, moved(x), 2, True))


@pytest.mark.parametrize("T,H,I,fmt", [(1, 8, 1 << 20, "bf16"), (2, 1 << 20, 8, "bf16"), (1, 32, (1 << 20) - 32, "nvfp4"),
                                       (9, 1 << 20, 32, "mxfp4"), (3, 1 << 20, 32, "nvfp4")])
def test_largest_widths(dev, T, H, I, fmt):
    layer = Layer(1, H, I, fmt, dev, 16)
    logits, x = tokens(T, 1, H, dev, 17)
    run_and_check(layer, logits, x, 1, False, f"T={T} H={H} I={I} {fmt}")


def test_new_memory_with_a_stream_of_its_own(dev):
    """Results and workspace of a call on another stream: not memory that the
    current stream still writes."""
    layer = Layer(8, 256, 128, "bf16", dev, 18)
    logits, x = tokens(4, 8, 256, dev, 19)
    want = layer(logits, x, 2, True)
    s = torch.cuda.Stream()
    slow = torch.randn(4096, 4096, device=dev)
    torch.cuda.synchronize()
    for _ in range(20):
        slow = (slow @ slow).clamp_(-1, 1)                             # the current stream is busy
        freed = [torch.empty_like(want).fill_(9) for _ in range(4)]   # written when its turn comes
        del freed
        got = layer(logits, x, 2, True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


FIRST = """
import torch
from memory_bound_moe_gb300 import moe_add_rmsnorm, moe_gemv_fp4, moe_layer, moe_layer_fp4
dev = torch.device("cuda:0")
T, E, H, I = 4, 8, 128, 64
bf = lambda *s: torch.randn(*s, device=dev).to(torch.bfloat16)
u8 = lambda *s: torch.randint(1, 100, s, device=dev, dtype=torch.uint8)
x, logits, w13, w2 = bf(T, H), torch.randn(T, E, device=dev), bf(E, 2 * I, H), bf(E, H, I)
q = (u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 16), u8(E, H, I // 2), u8(E, H, I // 16))
g = torch.ones(E, device=dev)
def step():
    return (moe_add_rmsnorm(x, None, w2[0, :, 0].contiguous())[0], moe_gemv_fp4(x, q[0][0], q[1][0]),
            moe_layer(logits, x, w13, w2, 2, True), moe_layer_fp4(logits, x, *q, 2, True, "nvfp4", g, g))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
eager = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
print("same")
"""


def test_first_calls_inside_a_capture(dev):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_back_to_back_calls_that_feed_each_other(dev):
    """Every call reads the previous one's output (x and, through a product,
    the logits): launches that overlap must not read early."""
    E, H, I, T, k = 16, 256, 128, 4, 4
    layer = Layer(E, H, I, "bf16", dev, 8)
    logits, x = tokens(T, E, H, dev, 9)
    router = (torch.randn(E, H, device=dev) / 16)

    def chain(sync):
        h, l = x, logits
        for _ in range(20):
            h = layer(l, h, k, True)
            if sync:
                torch.cuda.synchronize()
            h = (h.float() / h.float().norm(dim=1, keepdim=True) * 16).to(torch.bfloat16)
            l = h.float() @ router.t()
        return h
    assert torch.equal(chain(False), chain(True))


def test_empty_batch(dev):
    layer = Layer(4, 64, 32, "mxfp4", dev, 1)
    logits, x = tokens(1, 4, 64, dev, 1)
    assert layer(logits[:0], x[:0], 2, True).shape == (0, 64)
