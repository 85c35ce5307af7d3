"""Host-side refusals of the norm, cache, attention and routing calls: bad
arguments return the documented status (or raise in the binding) before
anything is enqueued; no GPU is touched."""
import pytest
import torch

from dequant_quantized_gemv_amd import qk

E = qk
W, X, Y, R, S, T, L, WS = (0x10000000 * i for i in range(1, 9))
BAD, UNSUP, ALIGN = E.QK_ERR_INVALID_ARG, E.QK_ERR_UNSUPPORTED, E.QK_ERR_ALIGNMENT


def _call(fn, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*a.values())


NORM = dict(xt=E.QK_F32, x=X, ldx=64, r=R, ldr=64, w=W, eps=1e-5, n=4, k=64, s=S, lds=64, yt=E.QK_F32, y=Y, ldy=64, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(xt=2), UNSUP), (dict(yt=3), UNSUP), (dict(xt=-1), UNSUP),
    (dict(n=-1), BAD), (dict(k=0), BAD), (dict(k=2 ** 30 + 1, ldx=2 ** 31, ldr=2 ** 31, lds=2 ** 31, ldy=2 ** 31), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(ldx=63), BAD), (dict(ldr=63), BAD), (dict(lds=63), BAD),
    (dict(ldy=63), BAD), (dict(yt=E.QK_X8, k=48), BAD), (dict(yt=E.QK_X8, ldy=71), BAD),
    (dict(yt=E.QK_X8, ldy=74), ALIGN), (dict(x=X + 2), ALIGN), (dict(r=R + 1), ALIGN), (dict(w=W + 2), ALIGN),
    (dict(y=Y + 2), ALIGN), (dict(s=S + 2), ALIGN), (dict(yt=E.QK_X8, ldy=72, y=Y + 2), ALIGN),
    (dict(y=X + 64), BAD), (dict(y=R + 64), BAD), (dict(y=W), BAD), (dict(y=S), BAD), (dict(s=W), BAD),
    (dict(s=X + 4), BAD), (dict(s=R, lds=65), BAD),
    (dict(n=0), E.QK_OK), (dict(n=0, x=None, y=None), E.QK_OK),
])
def test_norm_refusals(kw, want):
    assert _call(qk.qk_rms_norm, NORM, kw) == want


GEMV = dict(fmt=E.QK_Q8_0, w=W, m=8, k=64, x=X, n=2, ldx=72, y=Y, ldy=8, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=9), UNSUP), (dict(k=48), BAD), (dict(n=9), BAD), (dict(n=-1), BAD), (dict(m=-1), BAD),
    (dict(ldx=71), BAD), (dict(ldx=74), ALIGN), (dict(ldy=7), BAD), (dict(w=None), BAD), (dict(x=None), BAD),
    (dict(y=None), BAD), (dict(x=X + 2), ALIGN), (dict(w=W + 1), ALIGN), (dict(y=Y + 1), ALIGN), (dict(y=X + 140), BAD),
    (dict(y=W + 8), BAD), (dict(m=0), E.QK_OK), (dict(n=0), E.QK_OK), (dict(ldx=2 ** 62), BAD),
])
def test_x8q_refusals(kw, want):
    assert _call(qk.qk_mul_mat_vec_x8q, GEMV, kw) == want


def _desc(**kw):
    a = dict(type=E.QK_KV_I8, k=0x100000000, v=0x200000000, k_scale=0x300000000, v_scale=0x400000000, n_pages=8,
             n_heads=2, page_size=16, head_dim=64, page_stride=2048, head_stride=1024, slot_stride=64,
             scale_page_stride=32, scale_head_stride=16, scale_slot_stride=1)
    a.update(kw)
    return qk.KVCacheDesc(*a.values())


CACHES = [
    (dict(type=2), UNSUP), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD),
    (dict(n_pages=0), BAD), (dict(n_heads=0), BAD), (dict(page_size=0), BAD), (dict(head_dim=48), BAD),
    (dict(head_dim=0), BAD), (dict(head_dim=288), BAD), (dict(page_stride=-64), BAD), (dict(scale_slot_stride=-1), BAD),
    (dict(k=0x100000008), ALIGN), (dict(slot_stride=72), ALIGN), (dict(type=E.QK_KV_F16, slot_stride=68), ALIGN),
    (dict(k_scale=0x300000002), ALIGN), (dict(page_size=2 ** 21), BAD), (dict(page_stride=2 ** 62), BAD),
    (dict(n_pages=2 ** 31), BAD), (dict(n_heads=2 ** 20), BAD),
]

STORE = dict(k=X, k_tok=128, k_head=64, v=Y, v_tok=128, v_head=64, n=3, table=T, ldt=4, seqs=3, pages=4, seq=S, pos=L, stream=0)


@pytest.mark.parametrize("cache,kw,want", [(c, {}, w) for c, w in CACHES] + [
    (dict(slot_stride=48), {}, BAD), (dict(head_stride=512), {}, BAD), (dict(page_stride=1024), {}, BAD),  # rows meet
    (dict(scale_head_stride=8), {}, BAD), (dict(v=0x100000040), {}, BAD), (dict(v_scale=0x100000040), {}, BAD),
    ({}, dict(k=None), BAD), ({}, dict(v=None), BAD), ({}, dict(pos=None), BAD), ({}, dict(table=None), BAD),
    ({}, dict(n=-1), BAD), ({}, dict(ldt=3), BAD), ({}, dict(k_tok=-1), BAD), ({}, dict(k=X + 2), ALIGN),
    ({}, dict(pos=L + 2), ALIGN), ({}, dict(n=2 ** 30), BAD), ({}, dict(k=0x100000000), BAD),
    ({}, dict(table=0x300000000), BAD), ({}, dict(n=0), E.QK_OK),
])
def test_store_refusals(cache, kw, want):
    assert qk.qk_kv_store(_desc(**cache), *{**STORE, **kw}.values()) == want


def test_store_refuses_no_cache():
    assert qk.qk_kv_store(None, *STORE.values()) == BAD


ATTN = dict(q=X, q_seq=256, q_head=64, n=3, hq=4, table=T, ldt=4, lens=L, max_len=64, scale=0.125, window=0, sinks=0,
            yt=E.QK_F32, y=Y, y_seq=256, y_head=64, ws=None, wsb=0, stream=0)


@pytest.mark.parametrize("cache,kw,want", [(c, {}, w) for c, w in CACHES] + [
    ({}, dict(q=None), BAD), ({}, dict(y=None), BAD), ({}, dict(table=None), BAD), ({}, dict(lens=None), BAD),
    ({}, dict(n=-1), BAD), ({}, dict(hq=3), BAD), ({}, dict(hq=0), BAD), ({}, dict(ldt=3), BAD), ({}, dict(max_len=0), BAD),
    ({}, dict(max_len=2 ** 31), BAD), ({}, dict(window=-1), BAD), ({}, dict(sinks=-1), BAD), ({}, dict(yt=E.QK_X8), UNSUP),
    ({}, dict(y_head=63), BAD), ({}, dict(y_seq=255), BAD), ({}, dict(q=X + 2), ALIGN), ({}, dict(y=Y + 2), ALIGN),
    ({}, dict(lens=L + 1), ALIGN), ({}, dict(ws=WS + 8), ALIGN), ({}, dict(q_seq=-1), BAD), ({}, dict(y=X + 16), BAD),
    ({}, dict(y=T), BAD), ({}, dict(y=0x100000000), BAD), ({}, dict(y=0x400000000), BAD),
    ({}, dict(max_len=8192, ldt=512), BAD),                                # needs a workspace
    ({}, dict(max_len=8192, ldt=512, ws=WS, wsb=64), BAD),                 # a larger one
    ({}, dict(max_len=8192, ldt=512, ws=X, wsb=2 ** 30), BAD),             # not over q
    ({}, dict(n=0), E.QK_OK), ({}, dict(n=0, q=None, y=None, table=None, lens=None), E.QK_OK),
])
def test_attn_refusals(cache, kw, want):
    assert qk.qk_attn_decode(_desc(**cache), *{**ATTN, **kw}.values()) == want


def test_attn_workspace_sizes():
    assert qk.qk_attn_decode_workspace(_desc(), 3, 4, 64) == 0             # one chunk each
    assert qk.qk_attn_decode_workspace(_desc(), 3, 4, 8192) > 0
    assert qk.qk_attn_decode_workspace(_desc(), 3, 4, 8192, 32, 4) == 0    # a short window
    assert qk.qk_attn_decode_workspace(_desc(), 3, 3, 8192) == 0           # bad arguments
    assert qk.qk_attn_decode_workspace(_desc(k=None), 3, 4, 8192) == 0
    assert qk.qk_attn_decode_workspace(None, 3, 4, 8192) == 0


ROUTE = dict(x=X, ldx=64, n=3, e=64, used=8, score=E.QK_SIGMOID, bias=W, groups=8, kept=4, best=2, renorm=1, scale=1.0,
             ids=Y, ldi=8, w=S, ldw=8, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(score=2), UNSUP), (dict(n=-1), BAD), (dict(e=0), BAD), (dict(e=1025, ldx=1025, groups=1, kept=1), BAD),
    (dict(used=0), BAD), (dict(used=65), BAD), (dict(used=33), BAD), (dict(groups=0), BAD), (dict(groups=7), BAD),
    (dict(groups=128), BAD), (dict(kept=0), BAD), (dict(kept=9), BAD), (dict(best=0), BAD), (dict(best=3), BAD),
    (dict(x=None), BAD), (dict(ids=None), BAD), (dict(w=None), BAD), (dict(ldx=63), BAD), (dict(ldi=7), BAD),
    (dict(ldw=7), BAD), (dict(x=X + 2), ALIGN), (dict(ids=Y + 2), ALIGN), (dict(bias=W + 1), ALIGN),
    (dict(ids=X), BAD), (dict(w=X), BAD), (dict(ids=W), BAD), (dict(w=Y), BAD), (dict(n=0), E.QK_OK),
])
def test_route_refusals(kw, want):
    assert _call(qk.qk_moe_route, ROUTE, kw) == want


def test_binding_refusals():
    """The tensor wrappers raise before any launch (CPU tensors reach the
    device check last)."""
    f = torch.zeros
    with pytest.raises(TypeError):
        qk.rms_norm(f(2, 8, dtype=torch.float64))
    with pytest.raises(ValueError):
        qk.rms_norm(f(2, 40), out_dtype="x8")
    with pytest.raises(ValueError):
        qk.rms_norm(f(2, 8), out_dtype="bf16")
    with pytest.raises(ValueError):
        qk.rms_norm(f(2, 8), f(7))
    with pytest.raises(ValueError):
        qk.rms_norm(f(2, 8), residual_out=f(2, 8))
    with pytest.raises(TypeError):
        qk.rms_norm(f(2, 8), residual=f(2, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        qk.rms_norm(f(2, 8))
    with pytest.raises(TypeError):
        qk.mul_mat_vec_x8q("q4_0", f(18, dtype=torch.uint8), 1, 32, f(1, 36))
    with pytest.raises(ValueError):
        qk.mul_mat_vec_x8q("q4_0", f(18, dtype=torch.uint8), 1, 32, f(1, 35, dtype=torch.uint8))
    kv = [f(4, 2, 16, 64, dtype=torch.int8) for _ in range(2)]
    with pytest.raises(ValueError):
        qk.KVCache(*kv)
    with pytest.raises(TypeError):
        qk.KVCache(*kv, f(4, 2, 16, dtype=torch.float16), f(4, 2, 16, dtype=torch.float16))
    with pytest.raises(ValueError):
        qk.KVCache(*[f(4, 2, 16, 48, dtype=torch.float16) for _ in range(2)])
    with pytest.raises(ValueError):
        qk.KVCache(f(4, 2, 16, 64, dtype=torch.float16), f(4, 16, 2, 64, dtype=torch.float16).transpose(1, 2))
    with pytest.raises(TypeError):
        qk.KVCache(f(4, 2, 16, 64), f(4, 2, 16, 64))
    with pytest.raises(ValueError, match="CUDA"):
        qk.KVCache.empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError):
        qk.moe_route(f(2, 8), 2, score="tanh")
    with pytest.raises(TypeError):
        qk.moe_route(f(2, 8, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        qk.moe_route(f(2, 8), 65)
    with pytest.raises(ValueError):
        qk.moe_route(f(2, 8), 2, bias=f(7))
    with pytest.raises(ValueError, match="CUDA"):
        qk.moe_route(f(2, 8), 2)
