"""GPU: one workspace for the decode attention of a batch that shrinks and of
lengths below the bound that it was made for."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_one_workspace_serves_a_shrinking_batch(kind, window, sinks):
    t = torch()
    heads, hq, dim, page, most, seqs = 8, 16, 64, 16, 4096, 64
    rng = np.random.default_rng(1)
    pages = 300                                         # (shared: only the values count)
    shape = (pages, heads, page, dim)
    if kind == "f16":
        pools = [t.from_numpy(rng.standard_normal(shape).astype(np.float16)).cuda() for _ in range(2)]
    else:
        pools = [t.from_numpy(rng.integers(-127, 128, shape).astype(np.int8)).cuda() for _ in range(2)]
        pools += [t.from_numpy((rng.random(shape[:3]) * 0.02).astype(np.float32)).cuda() for _ in range(2)]
    cache = qk.KVCache(*pools)
    q = t.from_numpy(rng.standard_normal((seqs, hq, dim)).astype(np.float32)).cuda()
    table = t.from_numpy(rng.integers(0, pages, (seqs, most // page)).astype(np.int32)).cuda()
    lens = t.from_numpy(rng.integers(1, most + 1, seqs).astype(np.int32)).cuda()
    need = qk.qk_attn_decode_workspace(cache.desc, seqs, hq, most, window, sinks)
    guard = t.full((need + 4096,), 0xA5, dtype=t.uint8, device="cuda")
    for n in (64, 63, 56, 33, 20, 7, 1):
        for length in (4096, 4090, 2000, 1056, 1024, 130, 128):
            print("[case] shrinking batch", kind, window, n, length, flush=True)
            args = cache, q[:n], table[:n], lens[:n].clamp(max=length)
            y = qk.attn_decode(*args, max_len=length, window=window, sinks=sinks, workspace=guard[:need])
            assert t.equal(y, qk.attn_decode(*args, max_len=length, window=window, sinks=sinks)), (n, length)
            assert t.isfinite(y).all()
    assert (guard[need:] == 0xA5).all()
