"""GPU: the decode step of examples/moe_decode_step.py, which runs the norm,
the GEMVs, the cache store, the attention, the routing and the expert products
together, against the same step in 64 bits on the host.

Every step starts from the hidden states that the GPU step had.  The bound is on
the step's update (what it adds to the hidden states): 5e-3 of its rms, over
the update's entries.  fp32 leaves 1e-6; an 8-bit code that falls the other way
(a rounding that a tie turns on) is one step of about 40 in one of 512 entries
of a vector, 1e-3 of a product's rms.  A wrong operand anywhere is a sizeable
part of the update: attention and experts each make about half of it.
"""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu


def _norm(x, w):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w


def _x8(x):
    q, d = oracle.quantize_x8(np.ascontiguousarray(x, np.float32), x.shape[1], x.shape[0])
    n = x.shape[0]
    return (np.asarray(q, np.float64).reshape(n, -1, 32) * np.asarray(d, np.float64).reshape(n, -1, 1)).reshape(n, -1)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_decode_step_matches_64_bits(kind):
    from examples.moe_decode_step import main
    t = torch()
    record = []
    _, L, (past, seq, pos) = main(steps=3, kind=kind, time_it=False, record=record)
    t.cuda.synchronize()

    def dense(w, rows, k):
        return oracle.dequantize_f32(L.fmt, w.cpu().numpy(), rows, k).astype(np.float64).reshape(rows, k)

    wq, wk, wv = dense(L.wq, L.q_heads * L.dim, L.width), dense(L.wk, L.kv_heads * L.dim, L.width), dense(L.wv, L.kv_heads * L.dim, L.width)
    wo, wr = dense(L.wo, L.width, L.q_heads * L.dim), dense(L.wr, L.experts, L.width)
    gate, up = (dense(w, L.experts * L.inner, L.width).reshape(L.experts, L.inner, L.width) for w in (L.gate, L.up))
    down = dense(L.down, L.experts * L.width, L.inner).reshape(L.experts, L.width, L.inner)
    n1, n2, bias = (v.cpu().numpy().astype(np.float64) for v in (L.norm1, L.norm2, L.bias))

    def held(x):  # the values that the cache keeps
        if kind == "f16":
            return x.astype(np.float16).astype(np.float64)
        d = np.abs(x).max(-1, keepdims=True) / 127
        return np.rint(x / d) * d

    n = record[0][0].shape[0]
    rows = [[[], []] for _ in range(n)]
    for i, s in enumerate(seq.tolist()):
        for j in range(2):
            rows[s][j].append(held(past[j][i].cpu().numpy().astype(np.float64)))
    group = L.q_heads // L.kv_heads
    for x_in, x_out, now in record:
        x = x_in.cpu().numpy().astype(np.float64)
        h8 = _x8(_norm(x, n1))
        q, k, v = h8 @ wq.T, h8 @ wk.T, h8 @ wv.T
        att = np.zeros((n, L.q_heads * L.dim))
        for s in range(n):
            # the new token's place is one past those held: positions lens - 1
            for j, new in ((0, k), (1, v)):
                rows[s][j].append(held(new[s].reshape(L.kv_heads, L.dim)))
            K, V = np.stack(rows[s][0]), np.stack(rows[s][1])
            assert len(K) == int(now[s])
            for h in range(L.q_heads):
                z = K[:, h // group] @ q[s].reshape(L.q_heads, L.dim)[h] * L.dim ** -0.5
                p = np.exp(z - z.max())
                att[s, h * L.dim:(h + 1) * L.dim] = p @ V[:, h // group] / p.sum()
        x = att @ wo.T + x
        h = _norm(x, n2)
        p = 1 / (1 + np.exp(-(h @ wr.T)))
        val = p + bias
        g = np.sort(val.reshape(n, L.groups, -1), -1)[..., -2:].sum(-1)
        keep = np.argsort(-g, -1, kind="stable")[:, :L.groups // 2]
        y = np.zeros_like(x)
        for s in range(n):
            ok = np.isin(np.arange(L.experts) // (L.experts // L.groups), keep[s])
            ids = np.argsort(-np.where(ok, val[s], -np.inf), kind="stable")[:L.used]
            w = p[s][ids] / p[s][ids].sum()
            for e, we in zip(ids, w):
                a = gate[e] @ h[s]
                y[s] += we * (down[e] @ (a / (1 + np.exp(-a)) * (up[e] @ h[s])))
        want = x + y
        got = x_out.cpu().numpy().astype(np.float64)
        update = np.mean((want - x_in.cpu().numpy().astype(np.float64)) ** 2)
        off = np.sqrt(np.mean((got - want) ** 2) / update)
        print("[case] decode step", kind, off, np.sqrt(update), np.sqrt(np.mean(y ** 2)), flush=True)
        assert off < 5e-3


def test_decode_step_replayed_from_a_graph():
    """Every call of the step captured once and replayed: the eager bits."""
    from dequant_quantized_gemv_amd import qk
    from examples.moe_decode_step import Layer
    t = torch()
    layer = Layer()
    cache = qk.KVCache.empty(60, layer.kv_heads, 16, layer.dim, "i8")
    table = t.arange(60, dtype=t.int32, device="cuda").view(2, 30)
    g = t.Generator(device="cpu")
    g.manual_seed(5)
    for p in (cache.k, cache.v):
        p.copy_(t.randint(-127, 128, p.shape, generator=g).to(t.int8))
    for p in (cache.k_scale, cache.v_scale):
        p.copy_(0.01 * t.rand(p.shape, generator=g))
    lens = t.tensor([450, 17], dtype=t.int32, device="cuda")
    x = t.randn(2, layer.width, generator=g).cuda()
    ws = qk.attn_decode_workspace(cache, 2, layer.q_heads, 480)
    want = layer.step(x, cache, table, lens, ws)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            got = layer.step(x, cache, table, lens, ws)
    t.cuda.current_stream().wait_stream(s)
    for _ in range(4):
        got.fill_(float("nan"))
        if ws is not None:
            ws.fill_(255)
        layer.step(x * 0.5, cache, table, lens, ws)  # eager work between the replays
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(got, want)
