"""GPU: bounds of the decode attention that follow from how it holds its
values, and what a sequence's result does not depend on.

Per output, with A = sum_t p_t |V_t| / sum_t p_t and Z the largest over t of
scale * log2(e) * sum_i |q_i K_ti| (in 64 bits) and u = 2^-24: a score in log2 is
off by the two parts of q (2^-21 Z, and 2^-21 of the row's largest |q| times
scale * log2(e) * sum|K|), the sums over D products (D u Z) and four roundings
(4 u Z); a probability by ln2 times that and 2^-22 (exponential, and with 8 bits
its value's scale: it keeps its 24 bits and its exponent); numerator and
denominator: twice, and T sums (T u each).  Below 2^-126 nothing is held."""
import numpy as np
import pytest

from tests.gpu_helpers import torch
from tests.test_gpu_attn import Pages, _attn, _q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bound(pg, q, s, h, scale):
    """(y, bound) of one sequence and head."""
    x = q[s, h].astype(np.float64)
    K, V = (a[s][h * pg.heads // q.shape[1]] for a in (pg.k, pg.v))
    z = K @ x * scale
    p = np.exp(z - z.max())
    c = abs(scale) * 1.4426950408889634
    zz = (np.abs(K) @ np.abs(x)).max() * c
    zq = np.abs(K).sum(-1).max() * np.abs(x).max() * c
    dz = 2.0 ** -21 * (zz + zq) + (len(x) + 4) * U * zz
    a = p @ np.abs(V) / p.sum()
    return p @ V / p.sum(), (2 * (np.log(2) * dz + 2.0 ** -22) + (2 * len(K) + 8) * U) * a + 2.0 ** -126 * np.abs(V).sum(0)


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim,page,length,scale", [(32, 16, 9, 1e-3), (64, 16, 40, 0.02), (128, 24, 64, 0.0884),
                                                   (128, 16, 700, 1e-4), (256, 32, 33, 0.0625), (96, 16, 5, 1e-5)])
def test_probabilities_keep_their_bits(kind, dim, page, length, scale):
    """Small scores, so that what is left of the bound is the probabilities'."""
    print("[case] attn bounds", kind, dim, page, length, scale, flush=True)
    pg = Pages(kind, [length, length], 2, dim, page, dim + length)
    q = _q(2, 4, dim, length, 1.0)
    y = _attn(pg, q, scale=scale).astype(np.float64)
    for s in range(2):
        for h in range(4):
            want, bound = _bound(pg, q, s, h, scale)
            assert np.all(np.abs(y[s, h] - want) <= bound), (s, h)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_an_unlikely_token_decides_where_the_likely_ones_have_value_0(kind):
    """Value 0 at the likely tokens and one of probability 2^-20 .. 2^-100 of
    theirs with a value: the output has the bits of that probability."""
    t = torch()
    pg = Pages(kind, [50] * 5, 1, 64, 16, 3)
    q = np.ones((5, 1, 64), np.float32)
    pg.cache.k.zero_()
    if kind == "i8":
        pg.cache.k_scale.fill_(1.0 / 64)
    pg.cache.v.zero_()
    drop = [20, 40, 60, 80, 100]
    for s, n in enumerate(drop):
        pg.k[s][:] = 0
        pg.v[s][:] = 0
        at = int(pg.table[s, 2]), 0, 7                  # token 39
        pg.cache.k[at[0], 0, at[2], :32] = -2
        pg.k[s][0, 39, :32] = -2.0 if kind == "f16" else -2.0 / 64
        pg.cache.v[at[0], 0, at[2]] = t.arange(64, device="cuda").to(pg.cache.v.dtype)
        v = np.arange(64.0)
        if kind == "i8":
            v = v * float(pg.cache.v_scale[at])
        pg.v[s][0, 39] = v
        q[s] = n * np.log(2) / 64 * (1 if kind == "f16" else 64)
    y = _attn(pg, q, scale=1.0).astype(np.float64)
    for s in range(5):
        want, bound = _bound(pg, q, s, 0, 1.0)
        assert want[5] > 0 and np.all(np.abs(y[s, 0] - want) <= bound), drop[s]


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("length", [90, 5000])
def test_other_sequences_do_not_change_a_result(kind, length):
    """The same sequence beside others of other lengths, pages and values (as
    many of them, and the same bound on the lengths): the same bits."""
    t = torch()
    others = [[7, 0, 301], [length, 1, 64], [0, 0, 0]]
    got = []
    for i, lens in enumerate(others):
        pg = Pages(kind, [length] + lens, 2, 64, 16, 1, room=5120)
        rng = np.random.default_rng(i)
        q = rng.standard_normal((4, 4, 64)).astype(np.float32)
        q[0] = _q(1, 4, 64, 5)[0]
        got.append(_attn(pg, q)[0])
    # (the first draws of a seed's generator are the table and the values of all
    # pages, so that the first sequence holds the same)
    assert np.isfinite(got[0]).all()
    for y in got[1:]:
        assert np.array_equal(got[0].view(np.uint32), y.view(np.uint32))
