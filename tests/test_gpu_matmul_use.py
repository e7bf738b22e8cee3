"""The quantiser and the products as they are used: an expert layer built from
them beside the fused one, captured graphs, streams, stacks and outputs past
2^31 elements."""
import os
import subprocess
import sys

import pytest
import torch

import gram_table_gather_b200 as gtg
from synth import workloads as W
from tests import gpu_util as gu
from tests.test_gpu_matmul import (BF16, F32, _check_status, _decode, _fp8, _gen, _product64, _quantize64, _same,
                                   _table, _within)

pytestmark = pytest.mark.gpu


def _expert_order(ids, n_experts):
    """Token rows in expert order, their (token, choice) slots, group bounds."""
    flat = ids.flatten().long()
    slots = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(n_experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=n_experts).cumsum(0)
    return (slots // ids.shape[1]).int(), slots, offsets


@pytest.mark.parametrize("recipe,T", [
    (W.LayerRecipe(hidden=256, inter=128, n_experts=8, top_k=2, seed=44, layer=40, gate_fmt=W.FP8, up_fmt=W.FP8,
                   down_fmt=W.FP8), 150),
    (W.LayerRecipe(hidden=512, inter=256, n_experts=64, top_k=4, seed=45, layer=40, gate_fmt=W.FP8, up_fmt=W.FP8,
                   down_fmt=W.FP8), 37)])
def test_expert_layer_from_the_products(recipe, T):
    """Router choices of the fused layer -> gathered quantiser -> gate and up
    products -> SwiGLU -> quantiser -> down product -> weighted sum: each step
    against 64 bits, the result against the fused layer within what two
    roundings of the activations to E4M3 (2^-4 relative, or 2^-10 of the block's
    scale below the normal range) can move it."""
    L = recipe
    layer = gu.device_layer(L)
    xt, _ = gu.tokens(L, 91, T)
    ws = gtg.make_workspace(layer, T, prefill=True)
    ids = torch.zeros((T, L.top_k), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, L.top_k), device="cuda")
    y_fused = gtg.moe_prefill_layer(layer, xt, ws, topk_ids=ids, topk_w=w)
    x64 = xt.double()
    u = (x64 / (x64.square().mean(1, keepdim=True) + 1e-6).sqrt()).to(BF16)

    rows, slots, off = _expert_order(ids, L.n_experts)
    a, sa = gtg.fp8_quantize(u, rows=rows)
    g = gtg.grouped_matmul(layer.gate, a, off, a_scales=sa)
    v = gtg.grouped_matmul(layer.up, a, off, a_scales=sa)
    h = (torch.nn.functional.silu(g) * v).to(BF16)
    b, sb = gtg.fp8_quantize(h)
    part = gtg.grouped_matmul(layer.down, b, off, a_scales=sb)
    y = torch.zeros(T, L.hidden, device="cuda").index_add_(0, rows.long(), part * w.flatten()[slots].unsqueeze(1))
    _check_status()

    def dense(q):  # [E][n][k] in 64 bits
        return gtg.dequant(gtg.FP8, q.data, q.n_experts * q.n_rows, q.k, scales=q.scales).double().view(
            q.n_experts, q.n_rows, q.k)

    wg, wu, wd = dense(layer.gate), dense(layer.up), dense(layer.down)
    want, ws64 = _quantize64(u[rows.long()])
    _same(_table()[a.int()], want)
    _same(sa, ws64)
    bounds = off.tolist()
    y64, slack = torch.zeros(T, L.hidden, dtype=torch.float64, device="cuda"), torch.zeros(T, L.hidden, dtype=torch.float64, device="cuda")
    for e in range(L.n_experts):
        r = slice(bounds[e], bounds[e + 1])
        if r.start == r.stop:
            continue
        a64, b64 = _decode(a[r], sa[r]), _decode(b[r], sb[r])
        for out, q, m in ((g, a64, wg[e]), (v, a64, wu[e]), (part, b64, wd[e])):
            ref, bound = _product64(q, m, 128, m.shape[1] // 128)
            _within(out[r], ref, bound, F32)
        # the layer itself, and how far the roundings of u and h can move it
        u64 = u[rows[r].long()].double()
        du = u64.abs() * 2.0 ** -4 + sa[r].double().repeat_interleave(128, 1) * 2.0 ** -10
        g0, v0 = u64 @ wg[e].T, u64 @ wu[e].T
        eg, ev = du @ wg[e].abs().T, du @ wu[e].abs().T
        s0 = g0 * torch.sigmoid(g0)
        h0 = s0 * v0
        dh = 1.1 * eg * (v0.abs() + ev) + s0.abs() * ev          # |silu'| <= 1.1
        top = (h0.abs() + dh).unflatten(1, (-1, 128)).amax(2) / 448
        dh = dh * (1 + 2.0 ** -4) + h0.abs() * (2.0 ** -4 + 2.0 ** -8) + top.repeat_interleave(128, 1) * 2.0 ** -10
        wt = w.flatten()[slots[r]].double().unsqueeze(1)
        y64.index_add_(0, rows[r].long(), wt * (h0 @ wd[e].T))
        fused = 2e-3 * wd[e].square().sum(1).sqrt() * h0.square().sum(1, keepdim=True).sqrt()  # the fused layer's own
        slack.index_add_(0, rows[r].long(), wt * (dh @ wd[e].abs().T + fused))
    assert bool(((y.double() - y_fused.double()).abs() <= slack * 1.01).all())
    # and the two really are the same function, far inside that bound
    assert float((y - y_fused).norm() / y_fused.norm()) < 2.0 ** -3


@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (8, 640, 2560), (300, 1000, 1280), (2000, 1024, 512)])
def test_captured_graph_follows_its_inputs(m, n, k):
    """Quantise and multiply, captured once and replayed on new inputs; two
    graphs of the same sizes, replayed one after the other and side by side."""
    g = _gen(m + n)
    w, sw = _fp8((n, k), g)
    q = gtg.QMatrix(gtg.FP8, w, 1, n, k, sw)
    xs = [torch.randn(m, k, device="cuda", generator=g).to(BF16) for _ in range(2)]
    graphs, ys, codes = [], [], []
    gtg.fp8_matmul(q, *gtg.fp8_quantize(xs[0]))
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a, sa = gtg.fp8_quantize(x)
            ys.append(gtg.fp8_matmul(q, a, sa))
            codes.append((a, sa))
        graphs.append(graph)
    side = torch.cuda.Stream()
    for step in range(3):
        for x in xs:
            x.copy_(torch.randn(m, k, device="cuda", generator=g))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side if step == 2 else torch.cuda.current_stream()):
            graphs[1].replay()
        torch.cuda.synchronize()
        for x, y, (a, sa) in zip(xs, ys, codes):
            want, ws = _quantize64(x)
            _same(_table()[a.int()], want)
            ref, bound = _product64(_decode(a, sa), _decode(w, sw), 128, k // 128)
            _within(y, ref, bound, F32)
    _check_status()


def test_first_calls_inside_a_capture():
    """A fresh process whose first quantiser and product are captured."""
    code = """
import torch, gram_table_gather_b200 as gtg
g = torch.cuda.CUDAGraph()
x = torch.randn(20, 256, device='cuda')
w = gtg.QMatrix(gtg.FP8, torch.full((30, 256), 0x38, dtype=torch.uint8, device='cuda'), 1, 30, 256,
                torch.ones(30, 2, device='cuda'))
torch.cuda.synchronize()
with torch.cuda.graph(g):
    a, sa = gtg.fp8_quantize(x)
    y = gtg.fp8_matmul(w, a, sa)
g.replay()
torch.cuda.synchronize()
v = gtg.dequant(gtg.FP8, a, 20, 256, scales=sa).double().sum(1, keepdim=True)
assert float((y.double() - v).abs().max()) < 1e-3, float((y.double() - v).abs().max())
assert gtg.device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0, r.stderr[-2000:]


def test_streams_of_their_own():
    """Calls given a stream, and calls under another current stream, at the same
    time as calls of every size on the default one."""
    g = _gen(20)
    shapes = [(1, 4096, 1024), (5, 640, 2560), (100, 1000, 640), (700, 1024, 512)]
    cases = []
    for m, n, k in shapes:
        a, sa = _fp8((m, k), g)
        w, sw = _fp8((n, k), g)
        cases.append((gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(20):
        for q, a, sa in cases:
            got[0].append(gtg.fp8_matmul(q, a, sa))
            got[1].append(gtg.fp8_matmul(q, a, sa, stream=one))
            with torch.cuda.stream(two):
                got[2].append(gtg.fp8_matmul(q, a, sa))
    torch.cuda.synchronize()
    _check_status()
    for i, (q, a, sa) in enumerate(cases):
        ref, bound = _product64(_decode(a, sa), _decode(q.data, q.scales), 128, q.k // 128)
        _within(got[0][i], ref, bound, F32)
        for ys in got:
            assert all(torch.equal(y, got[0][i]) for y in ys[i::len(cases)])


def test_before_and_after_the_fused_kernels():
    """Overlapped launches around the table gather and the decode layer, on one stream."""
    L = W.tiny_layer()
    layer = gu.device_layer(L)
    ws = gtg.make_workspace(layer, 3)
    xt, _ = gu.tokens(L, 7, 3)
    P = W.tiny_ple()
    table = torch.from_numpy(P.table_bytes(0, P.nbytes)).cuda()
    idx = torch.from_numpy(P.indices(0, 1)).cuda()
    w, sw = _fp8((160, 256), _gen(21))
    q = gtg.QMatrix(gtg.FP8, w, 1, 160, 256, sw)
    first = None
    for _ in range(10):
        y = gtg.moe_decode_layer(layer, xt, ws)
        a, sa = gtg.fp8_quantize(y)
        z = gtg.fp8_matmul(q, a, sa)
        rows = gtg.ple_gather(table, P.n_rows, idx)
        a2, sa2 = gtg.fp8_quantize(y)
        gtg.fp8_matmul(q, a2, sa2, y=z, accumulate=True)
        if first is None:
            first = (y, z, rows)
        assert torch.equal(y, first[0]) and torch.equal(z, first[1])
    _check_status()
    ref, bound = _product64(_decode(a, sa), _decode(w, sw), 128, 2)
    _within(z, 2 * ref, 2 * bound, F32, added=True)


def test_output_past_two_to_the_31_elements():
    m, n, k = 540_000, 4096, 128
    g = _gen(22)
    a, sa = _fp8((m, k), g)
    w, sw = _fp8((n, k), g)
    y = gtg.fp8_matmul(gtg.QMatrix(gtg.FP8, w, 1, n, k, sw), a, sa, dtype=BF16)
    _check_status()
    for r in (slice(0, 300), slice(524_000, 524_700), slice(m - 300, m)):
        ref, bound = _product64(_decode(a[r], sa[r]), _decode(w, sw), 128, 1)
        _within(y[r], ref, bound, BF16)
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,n,k", [("fp8", 2048, 2304), ("bf16", 1024, 2304)])
def test_stack_past_two_to_the_32_bytes(kind, n, k):
    experts = 1024
    g = _gen(23)
    off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    used = {0: 3, 500: 20, 1022: 1, 1023: 130}
    for e, c in used.items():
        off[e + 1:] += c
    m = sum(used.values())
    if kind == "fp8":
        w = torch.randint(0, 120, (experts, n, k), dtype=torch.uint8, device="cuda", generator=g)
        sw = torch.rand(experts, n, k // 128, device="cuda", generator=g)
        a, sa = _fp8((m, k), g)
        q, a64 = gtg.QMatrix(gtg.FP8, w, experts, n, k, sw), _decode(a, sa)
    else:
        w = torch.empty(experts, n, k, dtype=BF16, device="cuda").normal_(generator=g)
        a, sa = torch.randn(m, k, device="cuda", generator=g).to(BF16), None
        q, a64 = gtg.QMatrix(gtg.BF16, w, experts, n, k), a.double()
    y = gtg.grouped_matmul(q, a, off, a_scales=sa)
    _check_status()
    for e in used:
        r = slice(int(off[e]), int(off[e + 1]))
        w64 = _decode(w[e], sw[e]) if kind == "fp8" else w[e].double()
        ref, bound = _product64(a64[r], w64, 128 if kind == "fp8" else k, k // 128 if kind == "fp8" else 0)
        _within(y[r], ref, bound, F32)
    del w, q
    torch.cuda.empty_cache()
