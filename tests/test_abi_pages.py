"""Host-side refusals of the calls on pages and page tables and of the log
probabilities: bad arguments return the documented status (or raise in the
binding) before anything is enqueued; no GPU is touched."""
import pytest
import torch

from dequant_quantized_gemv_amd import qk

E = qk
A, B, C, D, F, G, H, I, J, WS = (0x10000000 * i for i in range(1, 11))
BAD, UNSUP, ALIGN, OK = E.QK_ERR_INVALID_ARG, E.QK_ERR_UNSUPPORTED, E.QK_ERR_ALIGNMENT, E.QK_OK


def _call(fn, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*a.values())


def _desc(**kw):
    a = dict(type=E.QK_KV_I8, k=0x100000000, v=0x200000000, k_scale=0x300000000, v_scale=0x400000000, n_pages=8,
             n_heads=2, page_size=16, head_dim=64, page_stride=2048, head_stride=1024, slot_stride=64,
             scale_page_stride=32, scale_head_stride=16, scale_slot_stride=1)
    a.update(kw)
    return qk.KVCacheDesc(*a.values())


COPY = dict(cache=None, src=A, dst=B, n=4, stream=0)


@pytest.mark.parametrize("cache,kw,want", [
    (dict(), dict(n=-1), BAD), (dict(), dict(n=2 ** 31), BAD), (dict(), dict(src=None), BAD), (dict(), dict(dst=None), BAD),
    (dict(), dict(src=A + 2), ALIGN), (dict(), dict(dst=B + 1), ALIGN), (dict(), dict(src=0x100000000), BAD),
    (dict(), dict(dst=0x300000000 + 1020), BAD), (dict(slot_stride=0), dict(), BAD), (dict(page_stride=1024), dict(), BAD),
    (dict(scale_head_stride=8), dict(), BAD), (dict(v=0x100000000), dict(), BAD), (dict(type=7), dict(), UNSUP),
    (dict(k=None), dict(), BAD), (dict(k=0x100000008), dict(), ALIGN), (dict(), dict(n=0, src=None, dst=None), OK),
])
def test_copy_refusals(cache, kw, want):
    assert _call(qk.qk_kv_copy, dict(COPY, cache=_desc(**cache)), kw) == want


def test_copy_without_a_cache():
    assert _call(qk.qk_kv_copy, COPY, {}) == BAD


FORK = dict(table=A, ld_table=8, lens=B, n_rows=4, in_pages=8, parent=C, new_lens=D, n_new=6, out_pages=9, page_size=16, n_pages=100,
            out=F, ld_out=9, src=G, dst=H, missing=I, ws=WS, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(n_rows=-1), BAD), (dict(n_new=-1), BAD), (dict(in_pages=-1), BAD), (dict(out_pages=-1), BAD),
    (dict(page_size=0), BAD), (dict(page_size=2 ** 20 + 1), BAD), (dict(n_pages=0), BAD), (dict(n_pages=2 ** 31), BAD),
    (dict(in_pages=2 ** 30 + 1, ld_table=2 ** 31), BAD), (dict(n_new=2 ** 20, out_pages=2 ** 12, ld_out=2 ** 12), BAD),
    (dict(ld_table=7), BAD), (dict(ld_out=8), BAD), (dict(ld_out=2 ** 40), BAD),
    (dict(table=None), BAD), (dict(lens=None), BAD), (dict(new_lens=None), BAD), (dict(out=None), BAD), (dict(src=None), BAD),
    (dict(dst=None), BAD), (dict(missing=None), BAD), (dict(ws=None), BAD), (dict(ws_bytes=463), BAD),
    (dict(table=A + 1), ALIGN), (dict(lens=B + 2), ALIGN), (dict(parent=C + 2), ALIGN), (dict(out=F + 1), ALIGN),
    (dict(missing=I + 2), ALIGN), (dict(ws=WS + 8), ALIGN),
    (dict(out=A), BAD), (dict(out=A, ld_out=8, out_pages=8, parent=None), BAD), (dict(src=F + 8), BAD), (dict(dst=G), BAD),
    (dict(missing=H + 4), BAD), (dict(src=WS), BAD), (dict(out=D), BAD), (dict(dst=C), BAD), (dict(missing=B), BAD), (dict(ws=A), BAD),
])
def test_fork_refusals(kw, want):
    assert _call(qk.qk_kv_fork, FORK, kw) == want


COMPACT = dict(table=A, ld_table=8, lens=B, n_rows=4, max_pages=8, page_size=16, n_pages=100, out=F, ld_out=8, src=G, dst=H, live=I,
               ws=WS, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(n_rows=-1), BAD), (dict(max_pages=-1), BAD), (dict(page_size=0), BAD), (dict(n_pages=0), BAD), (dict(ld_table=7), BAD),
    (dict(ld_out=7), BAD), (dict(table=None), BAD), (dict(lens=None), BAD), (dict(out=None), BAD), (dict(src=None), BAD),
    (dict(dst=None), BAD), (dict(live=None), BAD), (dict(ws=None), BAD), (dict(ws_bytes=400), BAD), (dict(out=F + 2), ALIGN),
    (dict(ws=WS + 4), ALIGN), (dict(out=A, ld_out=9), BAD), (dict(out=A + 4), BAD), (dict(src=H), BAD), (dict(live=G + 196), BAD),
    (dict(dst=A), BAD), (dict(src=B), BAD), (dict(ws=F), BAD),
])
def test_compact_refusals(kw, want):
    assert _call(qk.qk_kv_compact, COMPACT, kw) == want


def test_pages_workspace():
    assert qk.qk_kv_pages_workspace(-1, 5) == 0 and qk.qk_kv_pages_workspace(1, 0) == 0
    last = 0
    for rows, pages in ((0, 1), (1, 1), (1, 33), (5, 33), (5, 1000), (1025, 1000), (1025, 70000)):
        need = qk.qk_kv_pages_workspace(rows, pages)
        assert need % 16 == 0 and need >= last and need >= 4 * (pages + rows) + pages // 4
        last = need


LOGP = dict(xt=E.QK_F32, x=A, ldx=100, n=4, vocab=100, scale=1.0, ids=B, ld_ids=2, n_ids=2, lp=C, ld_lp=2, entropy=D, top=5, bi=F,
            ld_bi=5, b=G, ld_b=5, ws=None, ws_bytes=0, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(xt=E.QK_X8), UNSUP), (dict(xt=-1), UNSUP), (dict(n=-1), BAD), (dict(vocab=0), BAD), (dict(vocab=2 ** 30 + 1, ldx=2 ** 31), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(n_ids=-1), BAD), (dict(n_ids=2 ** 20 + 1), BAD), (dict(top=-1), BAD), (dict(top=65), BAD), (dict(vocab=4, top=5), BAD),
    (dict(x=None), BAD), (dict(ids=None), BAD), (dict(lp=None), BAD), (dict(bi=None), BAD), (dict(b=None), BAD),
    (dict(ldx=99), BAD), (dict(ld_ids=1), BAD), (dict(ld_lp=1), BAD), (dict(ld_bi=4), BAD), (dict(ld_b=4), BAD),
    (dict(x=A + 2), ALIGN), (dict(xt=E.QK_F16, x=A + 1), ALIGN), (dict(ids=B + 2), ALIGN), (dict(lp=C + 1), ALIGN), (dict(entropy=D + 2), ALIGN),
    (dict(bi=F + 2), ALIGN), (dict(b=G + 2), ALIGN), (dict(lp=A), BAD), (dict(entropy=A + 1596), BAD), (dict(bi=B), BAD), (dict(b=F), BAD),
    (dict(entropy=C), BAD), (dict(vocab=40000, ldx=40000), BAD), (dict(vocab=40000, ldx=40000, ws=WS, ws_bytes=8), BAD),
    (dict(vocab=40000, ldx=40000, ws=WS + 8, ws_bytes=10000), ALIGN), (dict(vocab=40000, ldx=40000, ws=A, ws_bytes=10000), BAD),
    (dict(vocab=40000, ldx=40000, ws=C, ws_bytes=10000), BAD), (dict(n=0), OK), (dict(n=0, x=None, ids=None), OK),
])
def test_logprobs_refusals(kw, want):
    assert _call(qk.qk_token_logprobs, LOGP, kw) == want


def test_logprobs_workspace():
    """One entry for each 32768 logits of a row that has more; enough for any
    smaller call."""
    assert qk.qk_token_logprobs_workspace(-1, 100, 1) == 0 and qk.qk_token_logprobs_workspace(1, 0, 1) == 0
    assert qk.qk_token_logprobs_workspace(1, 100, 65) == 0 and qk.qk_token_logprobs_workspace(1, 32768, 20) == 0
    for n in (1, 2, 512, 5000):
        for v, parts in ((32769, 2), (65536, 2), (65537, 3), (2 ** 21, 64)):
            for top in (0, 1, 64):
                assert qk.qk_token_logprobs_workspace(n, v, top) == n * parts * (16 + 8 * top)


def _cpu(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    cache = qk.KVCache.__new__(qk.KVCache)
    t, n = _cpu(3, 4), _cpu(3)
    for call in (lambda: qk.kv_fork(t.float(), n, n, 16, 10), lambda: qk.kv_fork(t, n.long(), n, 16, 10),
                 lambda: qk.kv_fork(t, n, n.float(), 16, 10), lambda: qk.kv_fork(t, n, n, 16, 10, parent=n.long()),
                 lambda: qk.kv_compact(t.float(), n, 16, 10), lambda: qk.kv_copy(cache, n.float(), n), lambda: qk.kv_copy(cache, n, None),
                 lambda: qk.token_logprobs(t), lambda: qk.token_logprobs(t.double()), lambda: qk.token_logprobs(t.float(), ids=n.long()),
                 lambda: qk.token_logprobs(None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: qk.kv_fork(t, n[:2], n, 16, 10), lambda: qk.kv_fork(n, n, n, 16, 10), lambda: qk.kv_fork(t, n, n, 0, 10),
                 lambda: qk.kv_fork(t, n, n, 16, 0), lambda: qk.kv_fork(t, n, n, 16, 10, parent=n[:2]),
                 lambda: qk.kv_fork(t, n, n, 16, 10, out=_cpu(2, 4)), lambda: qk.kv_fork(t.t(), _cpu(4), n, 16, 10),
                 lambda: qk.kv_fork(t, n, n, 16, 10),        # not on a GPU
                 lambda: qk.kv_compact(t, n, 16, 10, out=_cpu(3, 5)), lambda: qk.kv_compact(t, n, 16, 10),
                 lambda: qk.kv_copy(cache, n, n[:2]), lambda: qk.kv_pages_workspace(3, 0),
                 lambda: qk.token_logprobs(n.float()), lambda: qk.token_logprobs(t.float().t()), lambda: qk.token_logprobs(t.float(), top=5),
                 lambda: qk.token_logprobs(t.float(), top=-1), lambda: qk.token_logprobs(t.float(), scale=0.0),
                 lambda: qk.token_logprobs(t.float(), ids=_cpu(2)), lambda: qk.token_logprobs(t.float(), ids=_cpu(3, 1, 1)),
                 lambda: qk.token_logprobs(t.float())):
        with pytest.raises(ValueError):
            call()
