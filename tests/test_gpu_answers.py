"""GPU: many answers to one prompt, the calls together as a program makes them:
a prompt stored once, forked into answers, every step with room for the new
token, the pages written on copied, attention with the shared tokens read
once, log probabilities to choose by, beams that drop and fork answers, and
the pool packed in between.  Against attention in 64 bits over each answer's own
tokens, kept apart from any page."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch().tensor(x, dtype=torch().int32, device="cuda")


def _attention(k, v, q):
    """(heads, group) rows of q over tokens (n, heads, dim), 64 bits."""
    out = []
    for h in range(k.shape[1]):
        z = q[h] @ k[:, h].T / np.sqrt(k.shape[2])
        p = np.exp(z - z.max(-1, keepdims=True))
        out.append(p @ v[:, h] / p.sum(-1, keepdims=True))
    return np.stack(out)


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("prompt,page,answers,layers", [(70, 16, 5, 2), (64, 16, 3, 1), (333, 24, 20, 1), (5, 8, 4, 2)])
def test_answers_to_a_prompt(kind, prompt, page, answers, layers):
    print("[case]", kind, prompt, page, answers, layers, flush=True)
    t = torch()
    rng = np.random.default_rng([prompt, page, answers])
    heads, group, dim, vocab, steps = 2, 3, 64, 500, 2 * page + 3
    per = -(-(prompt + steps) // page)
    # (every answer may need all of its own pages, and twice over while they are copied)
    pool = per * (2 * answers + 2)
    caches = [qk.KVCache.empty(pool, heads, page, dim, kind) for _ in range(layers)]
    ws = qk.kv_pages_workspace(max(answers, 1) + 1, pool)
    scratch = qk.attn_decode_shared_workspace(caches[0], answers, heads * group, per * page)

    def rows(n):
        """n tokens' keys and values of each layer, as they will lie in the cache, 64 bits."""
        x = rng.standard_normal((layers, 2, n, heads, dim)).astype(np.float32)
        if kind == "f16":
            return x, x.astype(np.float16).astype(np.float64)
        d = (np.abs(x).max(-1, keepdims=True) / np.float32(127)).astype(np.float32)
        return x, np.rint(x / d).astype(np.float64) * d

    # the prompt, in a row of its own
    table, src, dst, missing = qk.kv_fork(_i32([[-1] * per]), _i32([0]), _i32([prompt]), page, pool, workspace=ws)
    assert missing.item() == 0 and src.item() == -1
    x, held = rows(prompt)
    for l, c in enumerate(caches):
        qk.kv_store(c, *[t.from_numpy(x[l, i]).cuda() for i in (0, 1)], table, t.arange(prompt, dtype=t.int32, device="cuda"),
                    seq=t.zeros(prompt, dtype=t.int32, device="cuda"))
    tokens = [[held[:, :, i] for i in range(prompt)] for _ in range(answers)]   # of each answer: (layers, 2, heads, dim)
    lens = [prompt]
    parent = [0] * answers
    starts, whole = _i32([0, answers]), _i32([prompt // page * page])
    copied = 0
    for step in range(steps):
        new = [lens[p] + 1 for p in parent]
        table, src, dst, missing = qk.kv_fork(table, _i32(lens), _i32(new), page, pool, parent=_i32(parent), workspace=ws)
        assert missing.item() == 0
        copied += int((src >= 0).sum())
        for c in caches:
            qk.kv_copy(c, src, dst)
        lens = new
        x, held = rows(answers)
        for a in range(answers):
            tokens[a] = tokens[a] + [held[:, :, a]]
        q = rng.standard_normal((answers, heads * group, dim)).astype(np.float32)
        qd, ld = t.from_numpy(q).cuda(), _i32(lens)
        for l, c in enumerate(caches):
            qk.kv_store(c, *[t.from_numpy(x[l, i]).cuda() for i in (0, 1)], table, ld - 1)
            y = qk.attn_decode_shared(c, qd, table, ld, starts, whole, max_len=per * page, workspace=scratch)
            y1 = qk.attn_decode(c, qd, table, ld, max_len=per * page)
            for a in range(answers):
                kv = np.stack(tokens[a])[:, l]
                want = _attention(kv[:, 0], kv[:, 1], q[a].reshape(heads, group, dim).astype(np.float64)).reshape(-1, dim)
                # (scores of a few units in fp32, weights that sum to 1: 2^-18 of the largest value is well past the bound)
                top = np.abs(kv[:, 1]).max()
                assert np.all(np.abs(y[a].cpu().numpy() - want) <= 2.0 ** -18 * top), (step, l, a)
                assert np.all(np.abs(y1[a].cpu().numpy() - want) <= 2.0 ** -18 * top), (step, l, a)
        # the answers' next tokens, by what is likeliest
        logits = t.from_numpy(rng.standard_normal((answers, vocab)).astype(np.float32)).cuda()
        lp, entropy, ids, best = qk.token_logprobs(logits, top=answers)
        assert np.array_equal(ids.cpu().numpy(), np.argsort(-logits.cpu().numpy(), 1, kind="stable")[:, :answers])
        if step % 3 == 2:
            # beams: answers are dropped and others forked
            order = np.argsort(-best[:, 0].cpu().numpy(), kind="stable")
            parent = sorted(int(order[i % max(1, answers // 2)]) for i in range(answers))
        else:
            parent = list(range(answers))
        tokens = [tokens[p] for p in parent]
        if step % 5 == 4:
            # the pool packed; the lists move the pages of every layer
            table, src, dst, live = qk.kv_compact(table, _i32(lens), page, pool, workspace=ws)
            for c in caches:
                qk.kv_copy(c, src, dst)
            held_pages = table[table >= 0].unique()
            assert live.item() == len(held_pages) and held_pages.max().item() == live.item() - 1
    assert copied > 0 or answers < 2 or prompt % page == 0


def test_two_graphs_and_two_streams():
    """A step captured twice, with scratch of its own each, replayed on two
    streams at once."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(3)
    cache = qk.KVCache.empty(400, 2, 16, 64)
    cache.k.normal_(generator=g)
    cache.v.normal_(generator=g)
    logits = t.randn(6, 70000, device="cuda", generator=g)

    def make(seed):
        g.manual_seed(seed)
        table = t.randperm(400, device="cuda", generator=g).to(t.int32)[:180].view(6, 30)
        lens, starts, shared = _i32([300 + i + seed for i in range(6)]), _i32([0, 2, 6]), _i32([100, 250])
        q = t.randn(6, 8, 64, device="cuda", generator=g)

        def step():
            f = qk.kv_fork(table, lens, lens + 1, 16, 400)
            c = qk.kv_compact(table, lens, 16, 400)
            y = qk.attn_decode_shared(cache, q, table, lens, starts, shared)
            return [*f, *c, y, *qk.token_logprobs(logits, top=7)[1:]]
        want = step()
        s = t.cuda.Stream()
        s.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(s):
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph, stream=s):
                got = step()
        t.cuda.current_stream().wait_stream(s)
        return graph, s, got, want, step   # (which holds the inputs)

    both = [make(1), make(2)]
    t.cuda.synchronize()
    for _ in range(5):
        for graph, s, got, _w, _i in both:
            for x in got:
                x.zero_()
        t.cuda.synchronize()
        for graph, s, _g, _w, _i in both:
            with t.cuda.stream(s):
                graph.replay()
        t.cuda.synchronize()
        for _gr, _s, got, want, _i in both:
            for x, w in zip(got, want):
                assert t.equal(x, w)
