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
