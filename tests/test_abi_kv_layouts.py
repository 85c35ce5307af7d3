"""Caches in one piece of memory whose keys and values meet are refused by the
store before anything is enqueued; no GPU is touched."""
import pytest

from dequant_quantized_gemv_amd import qk

K, SC = 0x100000000, 0x300000000


def _store(**kw):
    """Status of a store over 4 pages of 2 heads, 16 tokens, 64 elements."""
    a = dict(type=qk.QK_KV_I8, k=K, v=K + 2048, k_scale=SC, v_scale=SC + 128, n_pages=4, n_heads=2, page_size=16,
             head_dim=64, page_stride=4096, head_stride=1024, slot_stride=64, scale_page_stride=64,
             scale_head_stride=16, scale_slot_stride=1)
    a.update(kw)
    return qk.qk_kv_store(qk.KVCacheDesc(*a.values()), 0x10000000, 128, 64, 0x20000000, 128, 64, 3, 0x30000000, 4, 3, 4,
                          0x40000000, 0x50000000, 0)


@pytest.mark.parametrize("kw", [
    dict(v=K), dict(v=K + 1024), dict(v=K + 64), dict(v=K + 4096), dict(v=K + 2048 - 16), dict(v=K + 2048 + 64),
    dict(v=K + 3 * 4096), dict(v=K - 1024), dict(v=K + 32, slot_stride=96, head_stride=1536),
    dict(v_scale=SC), dict(v_scale=SC + 64), dict(v_scale=SC + 4), dict(v_scale=SC + 256), dict(v_scale=SC - 64),
    dict(v_scale=K + 64), dict(k_scale=K + 2048 + 4), dict(k_scale=K + 4096 - 4),
    dict(type=qk.QK_KV_F16, v=K + 2048), dict(type=qk.QK_KV_F16, v=K + 8192),
])
def test_store_refuses_keys_and_values_that_meet(kw):
    assert _store(**kw) == qk.QK_ERR_INVALID_ARG
