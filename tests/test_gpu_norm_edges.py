"""GPU: qk_rms_norm where its factor leaves fp32's range, and 8-bit codes that
meet exact ties.  The bound is the norm's own: with u = 2^-24, |y - y64| <= 6 u
|y64| for fp32 outputs and half an ulp of the fp16 value more for fp16 ones."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _norm(x, eps, out="f32", weight=None):
    t = torch()
    w = None if weight is None else t.from_numpy(weight).cuda()
    return qk.rms_norm(t.from_numpy(x).cuda(), w, eps, out_dtype=out).cpu().numpy()


def _exact(x, eps):
    x = x.astype(np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


@pytest.mark.parametrize("k", [32, 200, 4096, 20000])
@pytest.mark.parametrize("out", ["f32", "f16"])
def test_rows_at_the_ends_of_fp32_without_eps(k, out):
    """Values down to one subnormal step and up to the largest float: the
    outputs are as near 1 as those of any other row."""
    rng = np.random.default_rng(k)
    unit = rng.standard_normal((9, k))
    x = (unit / np.abs(unit).max(-1, keepdims=True)).astype(np.float32)
    for i, scale in enumerate((1e-44, 1e-42, 1e-40, 2e-39, 1e-38, 1e-37, 1e37, 1e38, 3.4e38)):
        x[i] *= np.float32(scale)
    x[0, 0] = 1e-44                                     # (7 steps; the others may be 0)
    want = _exact(x, 0.0)
    y = _norm(x, 0.0, out).astype(np.float64)
    tol = 6 * U * np.abs(want) + (0 if out == "f32" else 2.0 ** -11 * np.abs(want) + 2.0 ** -25)
    assert np.all(np.abs(y - want) <= tol)


def test_one_subnormal_step_in_a_long_row():
    k = 1 << 20
    x = np.zeros((2, k), np.float32)
    x[0, 12345] = 2.0 ** -149
    x[1, 777] = -3.4e38
    y = _norm(x, 0.0).astype(np.float64)
    assert np.all(np.abs(y - _exact(x, 0.0)) <= 6 * U * np.abs(_exact(x, 0.0)))


@pytest.mark.parametrize("eps", [1e-300, 5e-324, 1e-60, 1e-78, 1e-100, 1e-115])
def test_zero_rows_with_a_tiny_eps_are_zero(eps):
    x = np.zeros((3, 96), np.float32)
    x[1] = 2.0 ** -149
    y = _norm(x, eps)
    assert not y[0].any() and not y[2].any()
    want = _exact(x[1:2], eps)
    # below fp32's smallest normal value, half a step
    assert np.all(np.abs(y[1] - want) <= 6 * U * want + 2.0 ** -150)


@pytest.mark.parametrize("scale", [2e-40, 1e38])
def test_8_bit_outputs_at_the_ends_of_fp32(scale):
    rng = np.random.default_rng(5)
    x = (rng.uniform(-1, 1, (2, 128)) * scale).astype(np.float32)
    y = _norm(x, 0.0)
    b = _norm(x, 0.0, "x8").reshape(2, 4, 36)
    d = b[..., :4].copy().view(np.float32)[..., 0]
    e = np.ceil(np.log2(np.abs(y).reshape(2, 4, 32).max(-1) / 127))
    assert np.array_equal(d, np.exp2(e).astype(np.float32))
    assert np.array_equal(b[..., 4:].view(np.int8), np.rint(y.reshape(2, 4, 32) / d[..., None]))


def test_8_bit_codes_round_ties_to_even():
    """Elements of magnitude 1 have the factor 1, so y is the weight: blocks
    of half-whole multiples of their scale."""
    k = 160
    w = np.zeros(k, np.float32)
    w[:32] = np.arange(32) - 15.5                       # largest 15.5, scale 2^-3: quotients whole
    w[32:64] = np.concatenate([[127.0], np.arange(31) - 15.5])            # scale 1
    w[64:96] = np.concatenate([[-126.5], np.arange(31) + 80.5])           # scale 1, large codes
    w[96:128] = np.concatenate([[100.0 * 2.0 ** 40], (np.arange(31) - 15.5) * 2.0 ** 40])
    w[128:] = np.concatenate([[127.0 * 2.0 ** -130], (np.arange(31) - 15.5) * 2.0 ** -126])
    x = np.where(np.arange(k) % 3 == 0, -1, 1).astype(np.float32)[None]
    b = _norm(x, 0.0, "x8", w).reshape(5, 36)
    d = b[:, :4].copy().view(np.float32)[:, 0].astype(np.float64)
    quotient = (x[0].astype(np.float64) * w).reshape(5, 32) / d[:, None]
    ties = np.abs(quotient - np.trunc(quotient)) == 0.5
    assert ties[1].sum() == 31 and ties[2].sum() == 32 and ties[3].sum() == 31 and ties[4].sum() == 31
    assert np.array_equal(d, [2.0 ** -3, 1, 1, 2.0 ** 40, 2.0 ** -126])
    assert np.array_equal(b[:, 4:].view(np.int8), np.rint(quotient))
