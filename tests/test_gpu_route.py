"""GPU: qk_moe_route through the C ABI, against the choice made in 64 bits.

Ids are compared exactly, on logits whose values in 64 bits lie more than 1e-5
apart (fp32 values are within 4 * 2^-24 of them, so no rounding can change the
order), and on exact ties.  Weights: an exponential (2 ulp), the sum (fp64,
rounded), a division, the sum of up to 64 and a division, so within 80 * 2^-24.
"""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import Guarded, torch

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, flush=True)


def _scores(x, score):
    x = x.astype(np.float64)
    if score == "sigmoid":
        return 1 / (1 + np.exp(-x))
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def _choose(x, used, score, bias=None, groups=1, kept=1, best=1, renorm=True, scale=1.0):
    """(ids, weights, least gap between neighbours in any ordered values)."""
    p = _scores(x, score)
    v = x.astype(np.float64) if bias is None and best == 1 else p + (0 if bias is None else bias.astype(np.float64))
    gap = np.diff(np.sort(v, -1), axis=-1).min() if v.shape[1] > 1 else np.inf
    if kept < groups:
        g = v.reshape(len(v), groups, -1)
        gs = np.sort(g, -1)[..., ::-1][..., :best].sum(-1)
        gap = min(gap, np.diff(np.sort(gs, -1), axis=-1).min())
        keep = np.argsort(-gs, -1, kind="stable")[:, :kept]
        in_kept = np.zeros_like(gs, bool)
        np.put_along_axis(in_kept, keep, True, -1)
        v = np.where(np.repeat(in_kept, v.shape[1] // groups, -1), v, -np.inf)
    ids = np.argsort(-v, -1, kind="stable")[:, :used]
    w = np.take_along_axis(p, ids, -1)
    if renorm:
        s = w.sum(-1, keepdims=True)
        w = np.where(s == 0, 0, w / np.where(s == 0, 1, s))
    return ids, w * scale, gap


def _logits(tokens, experts, seed, apart):
    """Random logits that `apart` accepts, row by row."""
    rng = np.random.default_rng(seed)
    rows = []
    while len(rows) < tokens:
        x = (rng.permutation(4 * experts)[:experts] / experts * 4 - 8 + rng.uniform(0, 0.2 / experts, experts))
        x = (x * 0.5).astype(np.float32)[None]
        if apart(x):
            rows.append(x)
    return np.concatenate(rows)


def _route(x, used, score, bias=None, groups=1, kept=1, best=1, renorm=True, scale=1.0, ldx=None, ldi=None, ldw=None):
    t = torch()
    n, experts = x.shape
    ldx, ldi, ldw = ldx or experts, ldi or used, ldw or used
    xd = t.full((n * ldx,), float("nan"), device="cuda")
    xd.as_strided((n, experts), (ldx, 1)).copy_(t.from_numpy(x.copy()))
    bd = t.from_numpy(bias.copy()).cuda() if bias is not None else None
    ids, w = Guarded(((n - 1) * ldi + used) * 4), Guarded(((n - 1) * ldw + used) * 4)
    st = qk.qk_moe_route(xd.data_ptr(), ldx, n, experts, used, {"softmax": 0, "sigmoid": 1}[score],
                         bd.data_ptr() if bd is not None else None, groups, kept, best, int(renorm), scale, ids.ptr,
                         ldi, w.ptr, ldw, t.cuda.current_stream().cuda_stream)
    assert st == qk.QK_OK, qk.status_string(st)
    i, v = ids.host(np.int32), w.host(np.float32)
    assert ids.guards_intact() and w.guards_intact()
    return (np.stack([i[r * ldi:r * ldi + used] for r in range(n)]),
            np.stack([v[r * ldw:r * ldw + used] for r in range(n)]))


CASES = [  # tokens, experts, used, groups, kept, best
    (1, 128, 8, 1, 1, 1), (1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 2), (5, 7, 3, 1, 1, 1), (17, 60, 6, 1, 1, 1),
    (33, 64, 8, 8, 3, 1), (9, 65, 4, 5, 2, 2), (40, 160, 6, 8, 3, 1), (13, 200, 16, 40, 7, 2), (21, 256, 8, 8, 4, 2),
    (6, 320, 64, 64, 40, 1), (4, 511, 9, 7, 5, 2), (5, 512, 8, 1, 1, 2), (3, 1024, 12, 16, 4, 2), (2, 64, 10, 64, 10, 2),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_route_matches_64_bits(score, biased, case):
    tokens, experts, used, groups, kept, best = case
    _say("route", score, biased, case)
    # (one value of 1024 softmax scores with a bias may lie near another: few experts are compared there)
    bias = np.random.default_rng(experts).permutation(experts).astype(np.float32) / 8 if biased else None
    kw = dict(bias=bias, groups=groups, kept=kept, best=best)

    def apart(x):
        return _choose(x, used, score, **kw)[2] > (1e-5 if biased or best == 1 else 1e-9)

    if not biased and best == 2:
        # scores alone, unsummed where groups == 1: keep the logits few steps
        # apart so that the scores differ in relative terms, which fp32 holds
        def apart(x):  # noqa: F811
            p = np.sort(_scores(x, score), -1)
            ok = experts == 1 or (np.diff(p, axis=-1) / p[:, 1:]).min() > 1e-5
            if kept < groups:
                g = np.sort(_scores(x, score).reshape(1, groups, -1), -1)[..., ::-1][..., :2].sum(-1)
                g = np.sort(g, -1)
                ok = ok and (np.diff(g, axis=-1) / g[:, 1:]).min() > 1e-5
            return ok
    x = _logits(tokens, experts, 1000 * experts + tokens, apart)
    ids, w = _route(x, used, score, **kw)
    rid, rw, _ = _choose(x, used, score, **kw)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 80 * 2.0 ** -24 * rw)


def test_route_strides_scale_and_plain_scores():
    x = _logits(11, 48, 4, lambda x: _choose(x, 5, "sigmoid")[2] > 1e-5)
    ids, w = _route(x, 5, "sigmoid", renorm=False, scale=2.5, ldx=53, ldi=9, ldw=6)
    rid, rw, _ = _choose(x, 5, "sigmoid", renorm=False, scale=2.5)
    assert np.array_equal(ids, rid) and np.all(np.abs(w - rw) <= 80 * 2.0 ** -24 * rw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [5, 64, 130, 700])
def test_route_ties_go_to_the_lowest_index(score, experts):
    x = np.zeros((3, experts), np.float32)
    x[1, ::2] = -0.0
    x[2, experts // 2:] = 1.0
    ids, w = _route(x, 4, score)
    assert np.array_equal(ids[:2], np.tile(np.arange(4), (2, 1)))
    assert np.array_equal(ids[2], experts // 2 + np.arange(4)[:max(0, experts - experts // 2)]
                          if experts - experts // 2 >= 4 else [2, 3, 4, 0])
    if experts > 5:
        assert np.allclose(w, 0.25)
    # equal groups: the first ones; equal values through a bias
    if experts % 5 == 0:
        kw = dict(groups=5, kept=2, best=2) if experts > 5 else dict(groups=5, kept=2, best=1)
        ids, _ = _route(x[:1], 2, score, bias=np.zeros(experts, np.float32), **kw)
        assert np.array_equal(ids[0], [0, 1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_and_non_finite_logits(score):
    """-inf logits (experts that are masked) come last, NaN after them; ids
    stay different; a row of -inf alone has weights 0 under softmax."""
    x = np.full((5, 70), -np.inf, np.float32)
    x[1, [3, 69]] = [1.0, 2.0]
    x[2, 5] = np.nan
    x[3] = np.arange(70)
    x[3, 69] = np.inf
    x[4] = np.nan
    ids, w = _route(x, 4, score)
    assert all(len(set(r)) == 4 and r.min() >= 0 and r.max() < 70 for r in ids)
    assert list(ids[0]) == [0, 1, 2, 3] and list(ids[1]) == [69, 3, 0, 1] and list(ids[2]) == [0, 1, 2, 3]
    assert list(ids[3]) == [69, 68, 67, 66] and list(ids[4]) == [0, 1, 2, 3]
    assert not w[0].any()                        # (sigmoid of -inf is 0 as well)
    ref = _choose(x[1:2], 4, score)[1]
    assert np.allclose(w[1], ref, rtol=80 * 2.0 ** -24, atol=0)
    if score == "softmax":
        assert np.isnan(w[2]).all() and np.isnan(w[3]).all()
    assert np.isnan(w[4]).all()
