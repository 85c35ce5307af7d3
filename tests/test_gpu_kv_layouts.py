"""GPU: caches whose keys and values lie in one tensor: the store and the
attention give what they give with pools of their own."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu
PAGES, HEADS, PAGE, DIM = 9, 3, 16, 64
# order of the dimensions (page, key or value, head, slot) in memory
ORDERS = ["pkhs", "kphs", "pskh", "phks", "pshk", "pksh", "spkh"]


def _pair(order, dtype, row, fill):
    """Keys and values as views (page, head, slot[, row]) of one tensor."""
    t = torch()
    size = {"p": PAGES, "k": 2, "h": HEADS, "s": PAGE}
    whole = t.full([size[d] for d in order] + ([row] if row else []), fill, dtype=dtype, device="cuda")
    at = order.index("k")
    rest = [d for d in order if d != "k"]
    views = []
    for i in range(2):
        v = whole.select(at, i)
        views.append(v.permute([rest.index(d) for d in "phs"] + ([3] if row else [])))
    return whole, views


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("order", ORDERS)
def test_keys_and_values_in_one_tensor(kind, order):
    print("[case] layout", kind, order, flush=True)
    t = torch()
    rng = np.random.default_rng(1)
    dtype = t.float16 if kind == "f16" else t.int8
    _, kv = _pair(order, dtype, DIM, 7)
    scales = _pair(order, t.float32, None, -1.0)[1] if kind == "i8" else []
    one = qk.KVCache(*kv, *scales)
    own = qk.KVCache(*[t.full((PAGES, HEADS, PAGE, DIM), 7, dtype=dtype, device="cuda") for _ in range(2)],
                     *[t.full((PAGES, HEADS, PAGE), -1.0, device="cuda") for _ in scales])
    tokens = 60
    k, v = (t.from_numpy(rng.standard_normal((tokens, HEADS, DIM)).astype(np.float32)).cuda() for _ in range(2))
    table = t.from_numpy(rng.permutation(PAGES)[:8].reshape(2, 4).astype(np.int32)).cuda()
    seq = t.arange(tokens, dtype=t.int32, device="cuda") % 2
    pos = t.arange(tokens, dtype=t.int32, device="cuda") // 2
    for c in (one, own):
        qk.kv_store(c, k, v, table, pos, seq=seq)
    for a, b in ((one.k, own.k), (one.v, own.v), (one.k_scale, own.k_scale), (one.v_scale, own.v_scale)):
        assert a is None or t.equal(a, b)
    q = t.from_numpy(rng.standard_normal((2, 2 * HEADS, DIM)).astype(np.float32)).cuda()
    lens = t.tensor([30, 25], dtype=t.int32, device="cuda")
    a, b = (qk.attn_decode(c, q, table, lens) for c in (one, own))
    # (scales that do not lie side by side are read token by token: other sums)
    assert t.equal(a, b) or t.allclose(a, b, rtol=0, atol=1e-5)
