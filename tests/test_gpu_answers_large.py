"""GPU: calls on pages, shared attention and log probabilities that go out in
several launches, and plans whose bits, lists or tables are past what one
workgroup holds in its first form."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch
from tests.test_gpu_pages import compact_reference, fork_reference

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, flush=True)


@pytest.mark.parametrize("n_pages", [131072, 262144, 262145])
def test_plans_of_large_pools(n_pages):
    """Around the largest pool that one workgroup plans."""
    _say("pool", n_pages)
    t = torch()
    rng = np.random.default_rng(n_pages)
    rows, per, page = 40, 1500, 16
    table = rng.permutation(n_pages)[:rows * per].reshape(rows, per).astype(np.int32)
    lens = rng.integers(0, per * page + 1, rows).astype(np.int32)
    new = np.minimum(lens + rng.integers(0, 200, rows), per * page).astype(np.int32)
    parent = rng.integers(-1, rows, rows).astype(np.int32)
    d = [t.from_numpy(x).cuda() for x in (table, lens, new, parent)]
    got = qk.kv_fork(d[0], d[1], d[2], page, n_pages, parent=d[3])
    for a, b in zip(got, fork_reference(table, lens, new, page, n_pages, parent, per)):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))
    got = qk.kv_compact(d[0], d[1], page, n_pages)
    for a, b in zip(got, compact_reference(table, lens, page, n_pages)):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


@pytest.mark.parametrize("n_pages", [20000, 16384, 9000, 4096, 1])
def test_many_pages_asked_for_at_once(n_pages):
    """Empty sequences given room: more requests than the list in LDS holds, and
    than there are pages."""
    _say("asked", n_pages)
    t = torch()
    rows, per, page = 64, 256, 16
    rng = np.random.default_rng(n_pages)
    table = rng.integers(0, n_pages, (rows, per)).astype(np.int32)
    lens = np.zeros(rows, np.int32)
    lens[3], lens[40] = 100, 33
    new = np.full(rows, per * page, np.int32)
    new[5], new[9] = 0, 17
    parent = np.full(rows, -1, np.int32)
    parent[3], parent[4], parent[40] = 3, 3, 40
    d = [t.from_numpy(x).cuda() for x in (table, lens, new, parent)]
    got = qk.kv_fork(d[0], d[1], d[2], page, n_pages, parent=d[3])
    for a, b in zip(got, fork_reference(table, lens, new, page, n_pages, parent, per)):
        assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


def test_copy_in_several_launches():
    """More workgroups than one launch takes, nearly all without a pair."""
    t = torch()
    cache = qk.KVCache.empty(9, 8, 16, 64)
    cache.k.normal_()
    cache.v.normal_()
    k, v = cache.k.clone(), cache.v.clone()
    n = 2_200_000   # 4 workgroups a pair
    src, dst = t.full((n,), -1, dtype=t.int32, device="cuda"), t.full((n,), -1, dtype=t.int32, device="cuda")
    for at, a, b in ((0, 1, 2), (2_097_151, 3, 4), (2_097_152, 0, 5), (n - 1, 7, 8)):
        src[at], dst[at] = a, b
        k[b], v[b] = k[a], v[a]
    qk.kv_copy(cache, src, dst)
    assert t.equal(cache.k, k) and t.equal(cache.v, v)


def test_log_probabilities_in_several_launches():
    t = torch()
    n = (1 << 25) + 100
    x = t.zeros(n, 2, device="cuda")
    x[:, 1] = t.arange(n, device="cuda") % 7 - 3.0
    ids = t.ones(n, dtype=t.int32, device="cuda")
    lp, entropy, best_ids, best = qk.token_logprobs(x, ids, top=1)
    want = t.log_softmax(x.double(), -1)
    assert t.allclose(lp.double(), want[:, 1], rtol=1e-6, atol=0)
    assert t.equal(best_ids[:, 0].bool(), x[:, 1] > 0)
    assert t.allclose(best[:, 0].double(), want.amax(-1), rtol=1e-6, atol=0)
    p = want.exp()
    assert t.allclose(entropy.double(), -(p * want).sum(-1), rtol=1e-6, atol=0)


def test_shared_attention_in_several_launches():
    """More workgroups of sequences' own tokens than one launch takes: every
    sequence sees one shared token and one of its own, or its own alone."""
    t = torch()
    n, heads, dim, page = 2_900_000, 3, 32, 1
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    cache = qk.KVCache.empty(1000, heads, page, dim)
    cache.k.normal_(generator=g)
    cache.v.normal_(generator=g)
    table = t.randint(0, 1000, (n, 2), device="cuda", generator=g).to(t.int32)
    half = n // 2
    starts, shared = (t.tensor(v, dtype=t.int32, device="cuda") for v in ([0, half], [1]))
    lens = t.ones(n, dtype=t.int32, device="cuda")
    lens[:half] = 2
    q = t.randn(n, heads, dim, device="cuda", generator=g)
    y = qk.attn_decode_shared(cache, q, table, lens, starts, shared, max_len=2, max_shared=1, max_own=1)
    for a, b in ((0, 5000), (half - 5000, half), (half, half + 5000), (n - 5000, n)):
        own = table[a:b, 1 if a < half else 0].long()
        k, v = cache.k[own][:, :, 0].double(), cache.v[own][:, :, 0].double()
        want = v
        if a < half:
            first = table[0, 0].long()
            z = t.stack([(q[a:b].double() * cache.k[first][:, 0].double()).sum(-1), (q[a:b].double() * k).sum(-1)], -1) / dim ** 0.5
            p = t.softmax(z, -1)
            want = p[..., :1] * cache.v[first][:, 0].double() + p[..., 1:] * v
        assert t.allclose(y[a:b].double(), want, rtol=0, atol=2.0 ** -18 * 8), (a, b)
