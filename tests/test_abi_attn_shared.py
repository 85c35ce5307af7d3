"""Host-side refusals of the attention with shared first tokens, and its
workspace; no GPU is touched."""
import pytest
import torch

from dequant_quantized_gemv_amd import qk

E = qk
Q, T, L, S, H, Y, WS = (0x10000000 * i for i in range(1, 8))
BAD, UNSUP, ALIGN, OK = E.QK_ERR_INVALID_ARG, E.QK_ERR_UNSUPPORTED, E.QK_ERR_ALIGNMENT, E.QK_OK


def _desc(**kw):
    a = dict(type=E.QK_KV_I8, k=0x100000000, v=0x200000000, k_scale=0x300000000, v_scale=0x400000000, n_pages=8,
             n_heads=2, page_size=16, head_dim=64, page_stride=2048, head_stride=1024, slot_stride=64,
             scale_page_stride=32, scale_head_stride=16, scale_slot_stride=1)
    a.update(kw)
    return qk.KVCacheDesc(*a.values())


ATTN = dict(cache=None, q=Q, q_seq=512, q_head=64, n_seqs=3, n_q_heads=8, table=T, ld_table=4, lens=L, max_len=64, starts=S, shared=H,
            n_groups=2, max_shared=40, max_own=30, scale=0.125, yt=E.QK_F32, y=Y, y_seq=512, y_head=64, ws=WS, ws_bytes=1 << 24, stream=0)


@pytest.mark.parametrize("cache,kw,want", [
    (dict(), dict(yt=E.QK_X8), UNSUP), (dict(type=5), dict(), UNSUP), (dict(head_dim=48), dict(), BAD), (dict(k_scale=None), dict(), BAD),
    (dict(), dict(n_seqs=-1), BAD), (dict(), dict(n_q_heads=7), BAD), (dict(), dict(n_q_heads=0), BAD), (dict(), dict(max_len=0), BAD),
    (dict(), dict(max_len=2 ** 30 + 1), BAD), (dict(), dict(n_groups=-1), BAD), (dict(), dict(n_groups=2 ** 31), BAD),
    (dict(), dict(max_shared=-1), BAD), (dict(), dict(max_shared=65), BAD), (dict(), dict(max_own=0), BAD), (dict(), dict(max_own=65), BAD),
    (dict(), dict(q=None), BAD), (dict(), dict(y=None), BAD), (dict(), dict(table=None), BAD), (dict(), dict(lens=None), BAD),
    (dict(), dict(starts=None), BAD), (dict(), dict(shared=None), BAD), (dict(), dict(ws=None), BAD), (dict(), dict(ws_bytes=1000), BAD),
    (dict(), dict(ld_table=3), BAD), (dict(), dict(q_seq=-1), BAD), (dict(), dict(y_head=32), BAD), (dict(), dict(y_seq=2 ** 28), BAD),
    (dict(), dict(q=Q + 2), ALIGN), (dict(), dict(starts=S + 1), ALIGN), (dict(), dict(shared=H + 2), ALIGN), (dict(), dict(y=Y + 2), ALIGN),
    (dict(), dict(ws=WS + 8), ALIGN), (dict(), dict(lens=L + 1), ALIGN),
    (dict(), dict(y=Q), BAD), (dict(), dict(y=WS), BAD), (dict(), dict(y=S), BAD), (dict(), dict(y=H), BAD), (dict(), dict(ws=T), BAD),
    (dict(), dict(ws=0x100000000), BAD), (dict(), dict(y=0x300000000), BAD), (dict(), dict(starts=WS + 16), BAD),
    (dict(), dict(n_seqs=0), OK), (dict(), dict(n_seqs=0, q=None, y=None, ws=None), OK),
])
def test_refusals(cache, kw, want):
    a = dict(ATTN, cache=_desc(**cache))
    a.update(kw)
    assert qk.qk_attn_decode_shared(*a.values()) == want


def test_without_a_cache():
    assert qk.qk_attn_decode_shared(*ATTN.values()) == BAD
    assert qk.qk_attn_decode_shared_workspace(None, 1, 8, 64, 10, 10) == 0


def _needed(heads, dim, seqs, q_heads, groups, max_shared, max_own):
    """Bytes of the partial results as the split is defined: per sequence and
    query head the chunks of shared tokens (enough for two workgroups per CU, one
    above head size 128, with the groups' row tiles) and those of its own (whole
    fours of 32-token tiles)."""
    target = 256 * (2 if dim <= 128 else 1)
    per = q_heads // heads
    n1 = 0
    if groups and max_shared:
        g = min(groups, seqs)
        each = -(-seqs * per // g)
        tiles = -(-max_shared // (128 if dim <= 64 else 64))
        for rows in ((128, 64) if each > 64 else (64,)):
            chunk = max(4 if tiles >= 32 else 1, min(tiles, -(-tiles * heads * g * -(-each // rows) // target)))
            if chunk * (1 if dim <= 128 else 2) >= 12:
                break
        n1 = -(-tiles // chunk)
    tiles = -(-(max_own + 31) // 32)
    rows = seqs * heads * -(-per // 16)
    chunk = min(tiles, max(4, -(-(-(-tiles * rows // target)) // 4) * 4))
    return 4 * seqs * q_heads * (n1 + -(-tiles // chunk)) * (dim + 4)


SEQS = [1, 2, 3, 8, 20, 31, 64, 100, 511, 1000]
SHARED = [0, 1, 64, 65, 1000, 8192, 131072]
OWN = [1, 33, 128, 1000, 12000]


@pytest.mark.parametrize("heads,q_heads,dim", [(8, 32, 128), (1, 1, 64), (8, 8, 192), (2, 34, 32), (1, 71, 96), (300, 300, 64)])
def test_one_workspace_serves_smaller_calls(heads, q_heads, dim):
    desc = qk.KVCacheDesc(qk.QK_KV_F16, 1 << 32, 1 << 40, None, None, 1000, heads, 16, dim, 16 * heads * dim, 16 * dim, dim, 0, 0, 0)
    need = {(n, s, o): max(_needed(heads, dim, n, q_heads, g, s, o) for g in (0, 1, 2, n // 3 + 1, n, 2 * n))
            for n in SEQS for s in SHARED for o in OWN}
    for n in SEQS:
        for s in SHARED:
            for o in OWN:
                asked = qk.qk_attn_decode_shared_workspace(desc, n, q_heads, 1 << 20, s, o)
                most = max(v for (a, b, c), v in need.items() if a <= n and b <= s and c <= o)
                assert asked >= most, (n, s, o, asked, most)


def _cpu(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    cache = qk.KVCache.__new__(qk.KVCache)
    cache.head_dim, cache.n_heads, cache.page_size = 64, 2, 16
    good = dict(q=_cpu(3, 4, 64, dtype=torch.float32), table=_cpu(3, 4), lens=_cpu(3), starts=_cpu(3), shared=_cpu(2))
    for kw in (dict(q=_cpu(3, 4, 64)), dict(q=None), dict(table=None), dict(lens=_cpu(3).long()), dict(starts=_cpu(3).float()), dict(shared=None)):
        with pytest.raises(TypeError):
            qk.attn_decode_shared(cache, **dict(good, **kw))
    for kw in (dict(starts=_cpu(2)), dict(lens=_cpu(2)), dict(table=_cpu(2, 4), lens=_cpu(2)), dict(q=_cpu(3, 3, 64, dtype=torch.float32)),
               dict(q=_cpu(3, 4, 32, dtype=torch.float32)), dict(max_len=65), dict(max_len=0), dict(max_shared=65), dict(max_shared=-1),
               dict(max_own=0), dict(max_own=65), dict(out_dtype="x8")):
        with pytest.raises(ValueError):
            qk.attn_decode_shared(cache, **dict(good, **kw))
