"""GPU: qk_token_logprobs against log-softmax in 64 bits.

Ids must be equal (a stable sort by the logit).  Tolerances, u = 2^-24, with d = S -
1 = the sum of exp(z) over all logits but one that is the largest:
  z in fp32: two roundings, and one for the factor log2(e) and its product
  each: 4u |z| in the exponent; the exponential 2u; sums of at most 64 terms in
  a thread, 6 exchanges, 8 waves, one rounding to fp32: 80u.  So d is within
  D = sum' exp(z) (4u |z| + 84u), and what is below fp32's range is lost: 2^-126 each.
  ln S: D / (1 + d).  A log probability adds its own rounding to fp32, u of it.
  The entropy's second term: sum exp(z) |z| (4u |z| + 2u + 84u) / S, and of its
  quotient D / (1 + d) of itself; then one rounding of the result.
"""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import Guarded, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _say(*a):
    print("[case]", *a, flush=True)


def reference(x, scale):
    """(log p, entropy, tolerance of ln S, tolerance of the entropy), 64 bits,
    of rows without NaN or +infinity."""
    x = x.astype(np.float64)
    n, vocab = x.shape
    lp, h, tl, th = np.full(x.shape, -np.inf), np.zeros(n), np.zeros(n), np.zeros(n)
    for r in range(n):
        m = x[r].max()
        if m == -np.inf:
            continue
        with np.errstate(under="ignore"):
            z = (x[r] - m) * scale
            e = np.exp(z)
        at = int(np.argmax(x[r]))
        rest = np.arange(vocab) != at
        az = np.where(e > 0, np.abs(z), 0.0)
        d = e[rest].sum()
        ln = np.log1p(d)
        lp[r] = z - ln
        w = (e * az).sum()
        h[r] = ln + w / (1 + d)
        dd = (e[rest] * (4 * U * az[rest] + 84 * U)).sum() + vocab * 2.0 ** -126
        tl[r] = dd / (1 + d)
        th[r] = tl[r] + (e * az * (4 * U * az + 86 * U)).sum() / (1 + d) + w / (1 + d) * tl[r] + vocab * 200 * 2.0 ** -126 + U * h[r]
    return lp, h, tl, th


def run(x, ids, top, scale=1.0, pad=0, offset=0):
    """Outputs through the C ABI, with guard bands; x fp32 or fp16."""
    t = torch()
    n, vocab = x.shape
    es = x.dtype.itemsize
    wide = np.full(offset + n * (vocab + pad) + 8, np.nan, x.dtype)
    ldx = vocab + pad
    for r in range(n):
        wide[offset + r * ldx:offset + r * ldx + vocab] = x[r]
    xd = t.from_numpy(wide).cuda()
    m = 0 if ids is None else ids.shape[1]
    idd = t.from_numpy(np.ascontiguousarray(ids, dtype=np.int32)).cuda() if m else None
    lp, h = Guarded(4 * n * (m + pad)), Guarded(4 * n)
    bi, b = Guarded(4 * n * (top + pad)), Guarded(4 * n * (top + pad))
    need = qk.qk_token_logprobs_workspace(n, vocab, top)
    ws = Guarded(need) if need else None
    st = qk.qk_token_logprobs(qk.QK_F32 if es == 4 else qk.QK_F16, xd.data_ptr() + es * offset, ldx, n, vocab, scale,
                              idd.data_ptr() if m else None, m, m, lp.ptr if m else None, m + pad, h.ptr, top,
                              bi.ptr if top else None, top + pad, b.ptr if top else None, top + pad, ws.ptr if ws else None, need)
    assert st == qk.QK_OK
    out = [g.host(dt).reshape(n, -1)[:, :k].copy() if n > 1 else g.host(dt)[:k].reshape(1, k).copy()
           for g, dt, k in ((lp, np.float32, m), (h, np.float32, 1), (bi, np.int32, top), (b, np.float32, top))]
    if n > 1 and pad:
        for g, k in ((lp, m), (bi, top), (b, top)):
            assert np.all(g.host(np.uint8).reshape(n, -1)[:, 4 * k:] == 0xA5)
    assert all(g.guards_intact() for g in [lp, h, bi, b] + ([ws] if ws else []))
    return out[0], out[1][:, 0], out[2], out[3]


def check(x, ids, top, scale=1.0, **kw):
    lp, h, best_ids, best = run(x, ids, top, scale, **kw)
    ref, rh, tl, th = reference(x, scale)
    n, vocab = x.shape

    def close(got, want, tol, what):
        want32 = np.abs(want)
        with np.errstate(invalid="ignore"):
            ok = (got == want) | (np.abs(got.astype(np.float64) - want) <= tol + U * want32 * (1 + 2.0 ** -20))
        assert np.all(ok), (what, got[~ok][:4], want[~ok][:4], np.broadcast_to(tol, got.shape)[~ok][:4])
    close(h, rh, th, "entropy")
    if ids is not None:
        inside = (ids >= 0) & (ids < vocab)
        want = np.take_along_axis(ref, np.clip(ids, 0, vocab - 1).astype(np.int64), 1)
        assert np.all(np.isnan(lp[~inside]))
        close(lp[inside], want[inside], np.broadcast_to(tl[:, None], ids.shape)[inside], "log probability")
    if top:
        order = np.argsort(-x.astype(np.float64), axis=1, kind="stable")[:, :top]
        assert np.array_equal(best_ids, order)
        close(best, np.take_along_axis(ref, order, 1), tl[:, None], "best")


VOCABS = [1, 2, 3, 7, 63, 64, 65, 511, 512, 513, 2047, 4095, 4096, 4097, 8191, 8193, 16384, 32000, 32768, 32769, 50257, 131073]


@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("vocab", VOCABS)
def test_vocabularies(vocab, dtype):
    _say("vocab", vocab, dtype.__name__)
    rng = np.random.default_rng(vocab)
    for n, top, m in ((1, min(20, vocab), 1), (3, min(5, vocab), 2), (2, 0, 0)):
        x = (rng.standard_normal((n, vocab)) * 3).astype(dtype)
        ids = rng.integers(0, vocab, (n, m)) if m else None
        check(x, ids, top, pad=0 if n == 1 else 5)


@pytest.mark.parametrize("n,vocab,top", [(600, 4097, 8), (1100, 1000, 1), (520, 32000, 5), (64, 20000, 64), (260, 33000, 64), (5, 262144, 20), (700, 33, 33)])
def test_rows(n, vocab, top):
    _say("rows", n, vocab, top)
    rng = np.random.default_rng(n)
    x = rng.standard_normal((n, vocab)).astype(np.float32)
    x[np.arange(n), rng.integers(0, vocab, n)] += rng.uniform(0, 30, n).astype(np.float32)
    check(x, rng.integers(0, vocab, (n, 3)), top, 1.25)


@pytest.mark.parametrize("scale", [0.01, 0.5, 1.0, 3.0, 1e-30, 1e30])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
def test_scales_and_offsets(scale, dtype):
    _say("scale", scale, dtype.__name__)
    rng = np.random.default_rng(7)
    for vocab in (100, 5001):
        x = (rng.standard_normal((3, vocab)) * 4).astype(dtype)
        for offset in (0, 1, 3):
            check(x, rng.integers(0, vocab, (3, 1)), 9, float(np.float32(scale)), pad=offset, offset=offset)


@pytest.mark.parametrize("vocab", [40, 5000, 40000])
def test_ties_go_to_the_lowest_index(vocab):
    _say("ties", vocab)
    rng = np.random.default_rng(vocab)
    for dtype in (np.float32, np.float16):
        for x in (np.zeros((2, vocab)), np.full((2, vocab), -2.5), rng.integers(0, 3, (2, vocab)), rng.integers(-40, 2, (3, vocab)),
                  np.where(rng.random((2, vocab)) < 0.5, 0.0, -0.0), np.arange(vocab)[None] // 7 * 1.0, -(np.arange(vocab)[None] // 9) * 1.0):
            check(x.astype(dtype) if vocab < 30000 or dtype == np.float32 else np.minimum(x, 60000).astype(dtype),
                  np.array([[0]] * len(x)), min(vocab, 64))


@pytest.mark.parametrize("vocab", [50, 4100, 40000])
@pytest.mark.parametrize("low", [-np.inf, -3.402823466e38, -1e30])
def test_masked_logits(vocab, low):
    """Masks that leave many, few, one or no tokens, at the row's ends and inside."""
    _say("masked", vocab, low)
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((7, vocab)).astype(np.float32)
    x[0, rng.random(vocab) < 0.5] = low
    keep = rng.integers(0, vocab, 10)
    x[1, np.setdiff1d(np.arange(vocab), keep)] = low
    x[2, 1:] = low
    x[3, :-1] = low
    x[4] = low
    x[5, :vocab // 2] = low
    x[6, vocab // 2:] = low
    check(x, np.stack([np.zeros(7, int), np.full(7, vocab - 1), np.full(7, keep[0])], 1), 20)


def test_one_token_has_nearly_all():
    """Log probabilities and entropies near 0 keep their digits."""
    for gap in (5.0, 16.0, 17.0, 30.0, 60.0, 87.0):
        x = np.zeros((1, 30000), np.float32)
        x[0, 123] = gap
        check(x, np.array([[123, 5]]), 3)
        lp, h, _, _ = run(x, np.array([[123]]), 0)
        d = 29999 * np.exp(-gap)
        assert abs(lp[0, 0] + np.log1p(d)) <= 1e-5 * np.log1p(d)
        assert abs(h[0] - (np.log1p(d) + gap * d / (1 + d))) <= 2e-5 * h[0]


@pytest.mark.parametrize("vocab", [5, 4500, 40000])
def test_nan_and_infinite_logits(vocab):
    _say("non-finite", vocab)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, vocab)).astype(np.float32)
    x[0, vocab // 2] = np.nan
    x[1, vocab - 1] = np.inf
    x[2] = np.nan
    x[3, :] = np.where(np.arange(vocab) % 2 == 0, np.nan, -np.inf)
    lp, h, ids, best = run(x, np.zeros((5, 1), int), 5)
    assert np.all(np.isnan(lp[:4])) and np.all(np.isnan(h[:4])) and np.all(np.isnan(best[:4]))
    for r in range(5):
        key = np.where(np.isnan(x[r]), -np.inf, x[r].astype(np.float64))
        order = sorted(range(vocab), key=lambda i: (bool(np.isnan(x[r, i])), -key[i], i))[:5]
        assert ids[r].tolist() == order, r
    check(x[4:], np.array([[0]]), 5)


def test_ids_outside_the_vocabulary():
    x = np.random.default_rng(1).standard_normal((2, 6000)).astype(np.float32)
    ids = np.array([[-1, 0, 5999, 6000], [2 ** 31 - 1, -2 ** 31, -100, 17]])
    check(x, ids, 3)


def test_binding_shapes_and_scratch():
    t = torch()
    x = t.randn(4, 33000, device="cuda")
    ids = t.randint(0, 33000, (4, 2), device="cuda", dtype=t.int32)
    lp, h, bi, b = qk.token_logprobs(x, ids, top=4)
    assert lp.shape == (4, 2) and h.shape == (4,) and bi.shape == b.shape == (4, 4)
    one, *_ = qk.token_logprobs(x, ids[:, 1].contiguous())
    assert one.shape == (4,) and t.equal(one, lp[:, 1])
    none = qk.token_logprobs(x)
    assert none[0] is None and none[2] is None and none[3] is None and t.equal(none[1], h)
    # scratch of larger calls serves, and holds nothing
    ws = qk.token_logprobs_workspace(64, 200000, 64)
    for fill in (0, 255):
        ws.fill_(fill)
        for a, c in zip(qk.token_logprobs(x, ids, top=4, workspace=ws), (lp, h, bi, b)):
            assert t.equal(a, c)
    # a part of a wider tensor
    wide = t.randn(4, 40000, device="cuda")
    part = wide[:, 5:30005]
    for a, c in zip(qk.token_logprobs(part, ids, top=2), qk.token_logprobs(part.contiguous(), ids, top=2)):
        assert t.allclose(a, c, rtol=0, atol=0, equal_nan=True)  # (ids behind the part's end: NaN)
    assert qk.token_logprobs(x[:0], ids[:0], top=3)[2].shape == (0, 3)


def test_in_a_graph():
    t = torch()
    x = t.empty(3, 50000, device="cuda")
    ids = t.zeros(3, 1, dtype=t.int32, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=s):
            got = qk.token_logprobs(x, ids, top=10)
    t.cuda.current_stream().wait_stream(s)
    for i in range(4):
        x.normal_()
        ids.random_(0, 50000)
        graph.replay()
        t.cuda.synchronize()
        for a, b in zip(got, qk.token_logprobs(x, ids, top=10)):
            assert t.equal(a, b), i
