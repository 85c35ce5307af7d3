"""GPU: the scores of qk_attn_decode_shared where every element of q is one fp16
part exactly: what is added to its low part of 0 (it must not be 0 beside an
infinite key) is no more than fp16's least value.

Tolerance of tests/test_gpu_attn_shared.py, in which the two parts of q cost
2^-21 of the row's largest; here 2^-37 of it: the least value, 2^-24, beside a
largest one of 2^13 at least.  So with A, Z and u as there
  scores: dz = 2^-37 max|q| sum|K| scale log2(e) + (D + 4) u Z in log2.
"""
import numpy as np
import pytest

from tests.gpu_helpers import torch
from tests.test_gpu_attn_shared import U, Batch, _say

pytestmark = pytest.mark.gpu
SCALE = float(np.float32(np.log(2)))   # times log2(e) it is 1 to fp32's last bit


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [3, 20, 40])
@pytest.mark.parametrize("seed", [0, 1])
def test_one_part_is_exact(dim, size, seed):
    _say("scores", dim, size, seed)
    t = torch()
    rng = np.random.default_rng([seed, dim, size])
    b = Batch("f16", [(size, 200)], [0] * size, 1, 2, dim, 16, seed=31)
    # a largest element beside which the others are small, keys that it does not
    # meet, large in every other token, and values of the sign that tells which
    shape = b.val["k"].shape
    large = np.arange(shape[2])[:, None] % 2
    k = np.round(rng.uniform(1500, 2048, shape) * large).astype(np.float16)
    k[..., 0] = 0
    v = (rng.uniform(0.5, 1, shape) * (2 * large - 1)).astype(np.float16)
    b.cache.k.copy_(t.from_numpy(k))
    b.cache.v.copy_(t.from_numpy(v))
    k, v = k.astype(np.float64), v.astype(np.float64)
    b.q = np.exp2(rng.integers(-20, -15, b.q.shape)).astype(np.float32)
    b.q[..., 0] = 1
    assert np.float32(SCALE * 1.4426950408889634) == 1
    got = b.run(scale=SCALE)
    for s in range(size):
        at = b.at[s]
        K, V = k[at[:, 0], 0, at[:, 1]], v[at[:, 0], 0, at[:, 1]]
        q = b.q[s].astype(np.float64)
        z = q @ K.T
        p = np.exp2(z - z.max(-1, keepdims=True))
        total = p.sum(-1, keepdims=True)
        want, A = p @ V / total, p @ np.abs(V) / total
        dz = 2.0 ** -37 * K.sum(-1).max() + (dim + 4) * U * z.max(-1, keepdims=True)
        tol = (2 * (np.log(2) * dz + 2.0 ** -22 + 2.0 ** -21) + 2 * len(K) * U + 9 * U) * A + 2.0 ** -36 * np.abs(V).sum(0) / total
        bad = ~(np.abs(got[s] - want) <= tol)
        assert not bad.any(), (s, got[s][bad][:5], want[bad][:5], tol[bad][:5], int(bad.sum()))
