"""GPU: keys that overflowed fp16.  A key of infinite score below zero has
probability 0 and the others share the sum; one above zero has no softmax."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu
LN2 = 0.69314718055994531


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("length", [20, 700, 9000])
def test_infinite_keys(page, length):
    """Queries whose halves are exact in fp16 (a power of two times a scale
    that is 1 in log2) and queries of all 24 bits; the infinities come in
    through the store."""
    print("[case] infinite keys", page, length, flush=True)
    t = torch()
    heads, hq, dim = 1, 4, 64
    rng = np.random.default_rng(length + page)
    per = -(-length // page)
    cache = qk.KVCache.empty(2 * per, heads, page, dim)
    k, v = (rng.standard_normal((length, heads, dim)).astype(np.float32) for _ in range(2))
    dead = rng.random(length) < 0.3
    dead[:3] = [False, True, True]
    k[dead, 0, 5] = -1e6                                # -inf in the cache
    table = t.arange(2 * per, dtype=t.int32, device="cuda").view(2, per)
    pos = t.arange(length, dtype=t.int32, device="cuda")
    kd, vd = t.from_numpy(k).cuda(), t.from_numpy(v).cuda()
    for s in range(2):
        qk.kv_store(cache, kd, vd, table, pos, seq=t.full((length,), s, dtype=t.int32, device="cuda"))
    q = np.zeros((2, hq, dim), np.float32)
    q[0] = np.exp2(rng.integers(-6, 1, (hq, dim))) * rng.choice([-1.0, 1.0], (hq, dim))
    q[1] = rng.standard_normal((hq, dim))
    q[..., 5] = np.abs(q[..., 5])
    q[0, 2] = 0
    q[0, 2, 5] = 1                                      # nothing but the infinite element
    lens = t.full((2,), length, dtype=t.int32, device="cuda")
    y = qk.attn_decode(cache, t.from_numpy(q).cuda(), table, lens, scale=LN2).cpu().numpy()
    K, V = k[~dead, 0].astype(np.float16).astype(np.float64), v[~dead, 0].astype(np.float16).astype(np.float64)
    for s in range(2):
        for h in range(hq):
            z = K @ q[s, h].astype(np.float64) * LN2
            p = np.exp(z - z.max())
            want = p @ V / p.sum()
            # the attention's bound: scores to (dim + 4) u and 2^-21 of sums of
            # magnitudes, probabilities 2^-22, sums of the tokens
            c = (np.abs(K) @ np.abs(q[s, h])).max() + np.abs(K).sum(-1).max() * np.abs(q[s, h]).max()
            rel = 2 * (LN2 * (2.0 ** -21 + (dim + 4) * 2.0 ** -24) * c + 2.0 ** -22) + (2 * len(K) + 8) * 2.0 ** -24
            assert np.all(np.abs(y[s, h] - want) <= rel * (p @ np.abs(V) / p.sum())), (s, h)
    # an infinite score above zero
    q[1, 3, 5] = -1.0
    y = qk.attn_decode(cache, t.from_numpy(q).cuda(), table, lens, scale=LN2).cpu().numpy()
    assert np.isnan(y[1, 3]).all() and np.isfinite(y[0]).all() and np.isfinite(y[1, :3]).all()


def test_rows_of_infinite_keys_alone_are_no_number():
    t = torch()
    cache = qk.KVCache(*[t.full((2, 1, 16, 64), float("-inf"), dtype=t.float16, device="cuda"),
                         t.ones((2, 1, 16, 64), dtype=t.float16, device="cuda")])
    table = t.tensor([[0, 1]], dtype=t.int32, device="cuda")
    q = t.ones(1, 2, 64, device="cuda")
    y = qk.attn_decode(cache, q, table, t.tensor([20], dtype=t.int32, device="cuda"))
    assert t.isnan(y).all()
