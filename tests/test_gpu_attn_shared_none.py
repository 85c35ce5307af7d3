"""GPU: qk_attn_decode_shared for a batch that shares nothing: no groups, or a
bound of 0 for what they share, at every head size.  Tolerance and reference
of tests/test_gpu_attn_shared.py."""
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch
from tests.test_gpu_attn_shared import Batch, _say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("groups", [[], [(3, 0)], [(2, 0), (0, 0), (1, -4)]])
def test_nothing_shared(kind, dim, groups):
    _say("none", kind, dim, groups)
    b = Batch(kind, groups, [1, 70, 33], 2, 3, dim, 16, seed=21)
    b.max_shared = 0
    b.check()
    b.check(bounds=(b.max_len, b.max_len, b.max_own))


def test_through_the_binding():
    t = torch()
    cache = qk.KVCache.empty(8, 2, 16, 128)
    cache.k.normal_()
    cache.v.normal_()
    table = t.arange(8, dtype=t.int32, device="cuda").view(2, 4)
    lens, starts = (t.tensor(x, dtype=t.int32, device="cuda") for x in ([60, 17], [0]))
    q = t.randn(2, 8, 128, device="cuda")
    want = qk.attn_decode(cache, q, table, lens)
    for kw in ({}, dict(max_shared=0)):
        y = qk.attn_decode_shared(cache, q, table, lens, starts, starts[:0], **kw)
        assert t.allclose(y, want, atol=1e-5, rtol=0)
