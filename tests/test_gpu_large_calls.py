"""GPU: calls whose threads together pass 2^32, which no one launch takes.  The
values are those of calls over parts of the same rows, bit for bit."""
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu
PART = 3 << 22  # rows; no divisor of a power of two


def test_norm_of_more_rows_than_a_launch_takes():
    t = torch()
    n, k = (1 << 26) + 5, 32
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    x = t.empty((n, k), dtype=t.float16, device="cuda")
    for i in range(0, n, PART):
        x[i:i + PART] = t.randn(min(PART, n - i), k, device="cuda", generator=g).half()
    w = t.randn(k, device="cuda", generator=g)
    for out in ("f16", "x8"):
        y = qk.rms_norm(x, w, out_dtype=out)
        for i in range(0, n, PART):
            assert t.equal(y[i:i + PART], qk.rms_norm(x[i:i + PART], w, out_dtype=out)), i
        del y
    # in place over the residual
    s = x.clone()
    y, _ = qk.rms_norm(x, w, residual=s, out_dtype="x8", residual_out=s)
    for i in range(0, n, PART):
        a, b = qk.rms_norm(x[i:i + PART], w, residual=x[i:i + PART], out_dtype="x8")
        assert t.equal(y[i:i + PART], a) and t.equal(s[i:i + PART], b), i


def test_route_of_more_tokens_than_a_launch_takes():
    t = torch()
    n, experts = (1 << 26) + 3, 3
    g = t.Generator(device="cuda")
    g.manual_seed(2)
    x = t.randn(n, experts, device="cuda", generator=g)
    ids, w = qk.moe_route(x, 2)
    for i in range(0, n, PART):
        a, b = qk.moe_route(x[i:i + PART], 2)
        assert t.equal(ids[i:i + PART], a) and t.equal(w[i:i + PART], b), i
    assert t.equal(ids[-3:].long(), x[-3:].sort(-1, descending=True)[1][:, :2])


@pytest.mark.parametrize("with_seq", [True, False])
def test_store_of_more_rows_than_a_launch_takes(with_seq):
    """64 heads of 32 elements: 2^23 tokens are 2^32 threads.  All tokens share
    one row of keys and one of values (strides of 0); most have no place, and
    the others lie at both ends and where parts of the call may meet."""
    t = torch()
    n, heads, dim, page = (1 << 23) + 70, 64, 32, 16
    places = [0, 1, 31, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 22) + 33, (1 << 23) - 1, 1 << 23, n - 2, n - 1]
    cache = qk.KVCache.empty(3, heads, page, dim)
    g = t.Generator(device="cuda")
    g.manual_seed(3)
    k, v = (t.randn(1, heads, dim, device="cuda", generator=g).expand(n, heads, dim) for _ in range(2))
    pos = t.full((n,), -1, dtype=t.int32, device="cuda")
    pos[places] = t.arange(len(places), dtype=t.int32, device="cuda") + 20
    if with_seq:
        table = t.tensor([[1, 2]], dtype=t.int32, device="cuda")
        seq = t.zeros(n, dtype=t.int32, device="cuda")
    else:
        table = t.tensor([1, 2], dtype=t.int32, device="cuda").repeat(n, 1)
        seq = None
    qk.kv_store(cache, k, v, table, pos, seq=seq)
    for x, pool in ((k, cache.k), (v, cache.v)):
        want = t.zeros_like(pool)
        for i in range(len(places)):
            want[table[0, (20 + i) // page].item(), :, (20 + i) % page] = x[0].half()
        assert t.equal(pool, want)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_attention_of_more_rows_than_a_launch_takes(kind):
    """2^21 sequences of 8 heads are 2^24 workgroups of 256.  All share a few
    pages, with lengths of 0 to 16 tokens."""
    t = torch()
    n, heads, dim, page, pages = (1 << 21) + 3, 8, 32, 16, 50
    g = t.Generator(device="cuda")
    g.manual_seed(4)
    shape = (pages, heads, page, dim)
    if kind == "f16":
        pools = [t.randn(*shape, device="cuda", generator=g).half() for _ in range(2)]
    else:
        pools = [t.randint(-127, 128, shape, device="cuda", dtype=t.int8, generator=g) for _ in range(2)]
        pools += [t.rand(shape[:3], device="cuda", generator=g) * 0.02 for _ in range(2)]
    cache = qk.KVCache(*pools)
    q = t.randn(n, heads, dim, device="cuda", generator=g)
    table = t.randint(0, pages, (n, 1), device="cuda", dtype=t.int32, generator=g)
    lens = t.randint(0, page + 1, (n,), device="cuda", dtype=t.int32, generator=g)
    y = qk.attn_decode(cache, q, table, lens)
    part = 300007
    for i in range(0, n, part):
        assert t.equal(y[i:i + part], qk.attn_decode(cache, q[i:i + part], table[i:i + part], lens[i:i + part])), i


def test_x8q_of_more_rows_than_a_launch_takes():
    """One block per row, two columns: the matrix-core kernel gives 16 rows a
    wave, so 2^30 rows are 2^32 threads."""
    t = torch()
    m, k = (1 << 30) + 37, 32
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    w = t.empty(m * 18, dtype=t.uint8, device="cuda")
    for i in range(0, m, PART):
        b = w[18 * i:18 * (i + PART)]
        b.random_(0, 256, generator=g)
        b.view(-1, 18)[:, :2] = t.tensor([0.0078125], dtype=t.float16, device="cuda").view(t.uint8)
    x = qk.rms_norm(t.randn(2, k, device="cuda", generator=g), out_dtype="x8")
    y = qk.mul_mat_vec_x8q("q4_0", w, m, k, x)
    for i in range(0, m, PART):
        rows = min(PART, m - i)
        part = qk.mul_mat_vec_x8q("q4_0", w[18 * i:18 * (i + rows)], rows, k, x)
        assert t.equal(y[:, i:i + rows], part), i
