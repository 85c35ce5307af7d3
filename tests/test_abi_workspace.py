"""The decode attention's workspace: what qk_attn_decode_workspace says for some
sizes serves every call of smaller ones.  The library's answers against the
split as it is defined, computed here; no GPU is touched."""
import pytest

from dequant_quantized_gemv_amd import qk

CUS = 256  # of the card; also what the library takes where there is none


def _desc(heads, dim):
    return qk.KVCacheDesc(qk.QK_KV_F16, 1 << 32, 1 << 40, None, None, 1000, heads, 16, dim, 16 * heads * dim, 16 * dim,
                          dim, 0, 0, 0)


def _asked(desc, seqs, q_heads, max_len, window=0, sinks=0):
    return qk.qk_attn_decode_workspace(desc, seqs, q_heads, max_len, window, sinks)


def _needed(heads, dim, seqs, q_heads, max_len, window=0, sinks=0):
    """Bytes of the partial results: one per sequence, query head and chunk;
    chunks of whole fours of 32-token tiles, two workgroups per CU (one above
    head size 128)."""
    tiles = -(-max_len // 32)
    if window:
        tiles = min(tiles, -(-min(sinks, max_len) // 32) + -(-min(window, max_len) // 32) + 1)
    rows = seqs * heads * -(-(q_heads // heads) // 16)
    target = CUS * (2 if dim <= 128 else 1)
    chunk = min(tiles, max(4, -(-(-(-tiles * rows // target)) // 4) * 4))
    chunks = -(-tiles // chunk)
    return 4 * seqs * q_heads * chunks * (dim + 4) if chunks > 1 else 0


SEQS = [1, 2, 3, 5, 8, 13, 20, 31, 33, 56, 63, 64, 100, 511, 512, 1000]
LENS = [1, 32, 128, 129, 160, 1000, 4096, 8192, 8224, 12000, 131072, 1 << 30]


@pytest.mark.parametrize("heads,q_heads,dim", [(8, 32, 128), (1, 1, 64), (8, 8, 192), (2, 34, 32), (5, 5, 256), (1, 71, 96),
                                               (300, 300, 64), (600, 600, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4), (5000, 300)])
def test_one_workspace_serves_smaller_calls(heads, q_heads, dim, window, sinks):
    desc = _desc(heads, dim)
    need = {(s, n): _needed(heads, dim, s, q_heads, n, window, sinks) for s in SEQS for n in LENS}
    for s in SEQS:
        for n in LENS:
            asked = _asked(desc, s, q_heads, n, window, sinks)
            assert asked >= max(v for (a, b), v in need.items() if a <= s and b <= n), (s, n)
            # and no more than twice the partial results that there can be workgroups for, or a row's own
            rows = heads * -(-(q_heads // heads) // 16)
            target = CUS * (2 if dim <= 128 else 1)
            assert asked <= 4 * q_heads * (dim + 4) * (target // rows + min(s, target // rows)), (s, n)


def test_a_shorter_window_needs_no_more():
    desc = _desc(8, 128)
    most = _asked(desc, 20, 32, 100000, 8000, 100)
    for window in (1, 31, 500, 1000, 1024, 4000, 7999):
        for sinks in (0, 4, 99):
            for seqs in (1, 7, 20):
                assert _needed(8, 128, seqs, 32, 50000, window, sinks) <= most
                assert _asked(desc, seqs, 32, 50000, window, sinks) <= most
