"""GPU: qk_rms_norm and qk_mul_mat_vec_x8q through the C ABI.

The norm against its formula in 64 bits.  With u = 2^-24: s is one rounding,
the factor one (its sum of squares in fp64 takes s as rounded: one more), the
two products one each, so |y - y64| <= 6 u |y64| for fp32 outputs, plus half an
ulp of the fp16 value for fp16 ones.  8-bit outputs are the blocks that the
oracle's quantization makes of the fp32 outputs, byte for byte.  The GEMV over
such blocks is held to the oracle's product as qk_mul_mat_vec_x8 is, and with
one column gives its bits.
"""
import numpy as np
import pytest

import oracle
from dequant_quantized_gemv_amd import qk, synth
from tests.gpu_helpers import D_RANGE, FMTS, Guarded, assert_within, to_dev_bytes, torch, x_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NP = {"f32": np.float32, "f16": np.float16}
CODE = {"f32": qk.QK_F32, "f16": qk.QK_F16, "x8": qk.QK_X8}


def _say(*a):
    print("[case]", *a, flush=True)


def _stream():
    return torch().cuda.current_stream().cuda_stream


def _inputs(n, k, xt, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((n, k)) * scale).astype(NP[xt])
    r = (rng.standard_normal((n, k)) * 2 * scale).astype(NP[xt])
    w = (1 + 0.3 * rng.standard_normal(k)).astype(np.float32)
    return x, r, w


def _norm(x, r, w, eps, xt, yt, ldx=None, ldy=None, x_off=0, y_off=0, want_sum=True):
    """(y as the stored bytes' rows, sum) of one call; guard bands checked."""
    n, k = x.shape
    es = np.dtype(NP[xt]).itemsize
    ldx = k if ldx is None else ldx
    row = k // 32 * 36 if yt == "x8" else k
    ye = 1 if yt == "x8" else np.dtype(NP[yt]).itemsize
    ldy = row if ldy is None else ldy
    hx, xp = x_dev(x, ldx, NP[xt], x_off)
    hr, rp = x_dev(r, ldx, NP[xt], x_off) if r is not None else (None, None)
    hw = torch().from_numpy(w).cuda() if w is not None else None
    y = Guarded(((n - 1) * ldy + row) * ye, y_off * (4 if yt == "x8" else ye))
    s = Guarded(((n - 1) * ldx + k) * es, x_off * es) if want_sum else None
    st = qk.qk_rms_norm(CODE[xt], xp, ldx, rp, ldx, hw.data_ptr() if hw is not None else None, eps, n, k,
                        s.ptr if s else None, ldx, CODE[yt], y.ptr, ldy, _stream())
    assert st == qk.QK_OK, qk.status_string(st)
    yb = y.host(np.uint8 if yt == "x8" else NP[yt])
    assert y.guards_intact()
    rows = np.stack([yb[j * ldy:j * ldy + row] for j in range(n)])
    sums = None
    if s:
        sb = s.host(NP[xt])
        assert s.guards_intact()
        sums = np.stack([sb[j * ldx:j * ldx + k] for j in range(n)])
        gaps = [sb[j * ldx + k:(j + 1) * ldx] for j in range(n - 1)]
        assert all(np.all(g.view(np.uint8) == 0xA5) for g in gaps), "sum wrote between rows"
    gaps = [yb[j * ldy + row:(j + 1) * ldy] for j in range(n - 1)]
    assert all(np.all(g.view(np.uint8) == 0xA5) for g in gaps), "y wrote between rows"
    return rows, sums


def _ref(x, r, w, eps):
    s = x.astype(np.float64) + (0 if r is None else r.astype(np.float64))
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s, y if w is None else y * w.astype(np.float64)


def _check(y, s, x, r, w, eps, xt, yt):
    s64, y64 = _ref(x, r, w, eps)
    half = 2.0 ** -11 * np.abs(y64) + 2.0 ** -25 if yt == "f16" else 0.0
    assert np.all(np.abs(y.astype(np.float64) - y64) <= 6 * U * np.abs(y64) + half + 1e-44)
    if s is not None:
        want = (x.astype(np.float32) + r.astype(np.float32)).astype(NP[xt])
        assert np.array_equal(s.view(np.uint8), want.view(np.uint8))


# rows below, at and past each kernel's reach; odd lengths with a tail of 1..3
@pytest.mark.parametrize("xt", ["f32", "f16"])
@pytest.mark.parametrize("yt", ["f32", "f16"])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 2), (5, 3), (1, 33), (7, 255), (4, 1024), (6, 1025), (1, 4096), (9, 4096),
                                 (3, 4099), (300, 5), (2, 11008), (2, 16384), (2, 16387), (1, 50001)])
def test_norm_matches_formula(xt, yt, n, k):
    _say("norm", xt, yt, n, k)
    x, r, w = _inputs(n, k, xt, 11 * n + k)
    y, s = _norm(x, r, w, 1e-5, xt, yt)
    _check(y, s, x, r, w, 1e-5, xt, yt)


@pytest.mark.parametrize("xt", ["f32", "f16"])
def test_norm_strides_offsets_and_absent_operands(xt):
    x, r, w = _inputs(5, 1030, xt, 3)
    for ldx, ldy, xo, yo in ((1031, 1033, 1, 1), (1100, 1030, 3, 2)):
        y, s = _norm(x, r, w, 1e-6, xt, "f32", ldx, ldy, xo, yo)
        _check(y, s, x, r, w, 1e-6, xt, "f32")
    y, _ = _norm(x, None, None, 1e-6, xt, "f32", want_sum=False)
    _check(y, None, x, None, None, 1e-6, xt, "f32")
    y, _ = _norm(x, r, None, 1e-6, xt, "f16", want_sum=False)
    _check(y, None, x, r, None, 1e-6, xt, "f16")


@pytest.mark.parametrize("yt", ["f32", "f16", "x8"])
def test_norm_sum_in_place(yt):
    """sum may be x or the residual itself, rows read twice among them."""
    t = torch()
    for k in (96, 4096, 16416):
        x, r, w = _inputs(3, k, "f32", k)
        for which in ("x", "r"):
            xd, rd, wd = (t.from_numpy(v.copy()).cuda() for v in (x, r, w))
            want, s = qk.rms_norm(xd, wd, residual=rd, out_dtype=yt)
            out = xd if which == "x" else rd
            y, _ = qk.rms_norm(xd, wd, residual=rd, out_dtype=yt, residual_out=out)
            assert t.equal(y, want) and t.equal(out, s), (yt, k, which)


def test_norm_extreme_rows():
    """Zero rows, rows whose squares leave fp32 either way, eps == 0."""
    x = np.zeros((5, 200), np.float32)
    x[1] = 1e30
    x[2] = 1e-30
    x[3, 7] = 3e38
    x[4] = np.arange(200) - 100
    y, _ = _norm(x, None, None, 1e-6, "f32", "f32", want_sum=False)
    _check(y[[0, 1, 3, 4]], None, x[[0, 1, 3, 4]], None, None, 1e-6, "f32", "f32")
    y, _ = _norm(x[1:], None, None, 0.0, "f32", "f32", want_sum=False)
    _check(y, None, x[1:], None, None, 0.0, "f32", "f32")
    # a zero row without eps is 0 / 0; an infinite or NaN element stays in its row
    x[2, 5], x[3, 6] = np.inf, np.nan
    y, _ = _norm(x, None, None, 0.0, "f32", "f32", want_sum=False)
    assert np.isnan(y[0]).all() and np.isnan(y[2, 5]) and np.isnan(y[3]).all()
    _check(y[[1, 4]], None, x[[1, 4]], None, None, 0.0, "f32", "f32")


@pytest.mark.parametrize("xt", ["f32", "f16"])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 96), (4, 1056), (1, 4096), (7, 4096), (2, 11008), (1, 16416)])
def test_norm_x8_is_the_quantized_fp32_output(xt, n, k):
    _say("norm x8", xt, n, k)
    x, r, w = _inputs(n, k, xt, 7 * n + k)
    x[0, :32] = 0
    r[0, :32] = 0                      # an all-zero block
    y, _ = _norm(x, r, w, 1e-5, xt, "f32")
    b, s = _norm(x, r, w, 1e-5, xt, "x8", ldy=k // 32 * 36 + 8)
    _check(y, s, x, r, w, 1e-5, xt, "f32")
    q, d = oracle.quantize_x8(y, k, n)
    got = b.reshape(n, k // 32, 36)
    assert np.array_equal(got[..., 4:].view(np.int8).reshape(n, k), np.asarray(q).reshape(n, k))
    assert np.array_equal(got[..., :4].copy().view(np.float32)[..., 0], np.asarray(d).reshape(n, k // 32))


def test_norm_x8_ties_and_non_finite_blocks():
    """A unit factor and exact ties; a block with an infinite value has a NaN
    scale and codes 0."""
    k = 96
    x = np.zeros((1, k), np.float32)
    x[0, :32] = (np.arange(32) - 16) + 0.5
    x[0, 32:64] = np.concatenate([[127.0], (np.arange(31) - 15) + 0.5])
    # the weight undoes the factor up to a power of two: codes meet exact ties
    s64 = np.sqrt((x.astype(np.float64) ** 2).mean())
    w = np.full(k, 1.0, np.float32)
    y, _ = _norm(x, None, w, 0.0, "f32", "f32", want_sum=False)
    b, _ = _norm(x, None, w, 0.0, "f32", "x8", want_sum=False)
    q, d = oracle.quantize_x8(y, k, 1)
    got = b.reshape(1, 3, 36)
    assert s64 > 0 and np.array_equal(got[..., 4:].view(np.int8).reshape(1, k), np.asarray(q).reshape(1, k))
    assert np.array_equal(got[..., :4].copy().view(np.float32).reshape(-1), np.asarray(d).reshape(-1))
    w[40] = np.inf
    b, _ = _norm(x, None, w, 0.0, "f32", "x8", want_sum=False)
    got = b.reshape(3, 36)
    dd = got[:, :4].copy().view(np.float32)[:, 0]
    assert np.isnan(dd[1]) and not np.isnan(dd[[0, 2]]).any()
    assert not got[1, 4:].any()


def _blocks(q, d):
    n, nb = d.shape
    b = np.zeros((n, nb, 36), np.uint8)
    b[..., :4] = np.ascontiguousarray(d.astype(np.float32))[..., None].view(np.uint8)
    b[..., 4:] = q.astype(np.int8).reshape(n, nb, 32).view(np.uint8)
    return b.reshape(n, nb * 36)


def _x8q(fmt, w, m, k, b, ldx=None, ldy=None, w_off=0, x_off=0):
    n, row = b.shape
    ldx = row if ldx is None else ldx
    ldy = m if ldy is None else ldy
    hw, wp = to_dev_bytes(w, w_off)
    hx, xp = x_dev(b, ldx, np.uint8, x_off)
    out = Guarded(((n - 1) * ldy + m) * 4)
    st = qk.qk_mul_mat_vec_x8q(fmt, wp, m, k, xp, n, ldx, out.ptr, ldy, _stream())
    assert st == qk.QK_OK, qk.status_string(st)
    y = out.host(np.float32)
    assert out.guards_intact()
    return np.stack([y[j * ldy:j * ldy + m] for j in range(n)])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,k,n", [(1, 32, 1), (3, 96, 2), (61, 544, 1), (100, 4096, 8), (259, 11008, 3),
                                   (33, 1376, 4), (17, 2048, 5), (8, 256, 7), (4097, 1024, 1), (700, 8224, 6),
                                   (50, 2112, 2), (4099, 4096, 3), (16, 4096, 8), (31, 4064, 4), (1, 11040, 8),
                                   (2000, 512, 4), (47, 1088, 8)])
def test_x8q_within_tolerance_and_one_column_as_x8(fmt, m, k, n):
    _say("x8q", fmt, m, k, n)
    w = synth.quant_matrix(fmt, m, k, seed=191, tensor_id=1, d_range=D_RANGE[fmt])
    x = synth.activations(k, n, seed=191, tensor_id=2)
    q, d = oracle.quantize_x8(x, k, n)
    y = _x8q(fmt, w, m, k, _blocks(np.asarray(q).reshape(n, k), np.asarray(d).reshape(n, k // 32)))
    t = torch()
    want = qk.mul_mat_vec_x8(fmt, t.from_numpy(w.copy()).cuda(), m, k, t.from_numpy(x.copy()).cuda()).cpu().numpy()
    assert n > 1 or np.array_equal(y.view(np.uint32), want.view(np.uint32))
    yref, s = oracle.dot_x8(fmt, w, m, k, x, n)
    assert_within(y, yref, s, 1e-4, f"x8q {fmt} {m}x{k} n={n}")


@pytest.mark.parametrize("fmt", FMTS)
def test_x8q_any_scales_strides_and_alignment(fmt):
    """Scales that are no powers of two, codes -128..127, 2-byte aligned
    weights, padded columns; against the product in 64 bits: per block one
    scaled term of an exact integer (three roundings, two such terms with an
    offset) and the fp32 sum over k/32 of them."""
    m, k, n = 45, 1056, 3
    rng = np.random.default_rng(5)
    w = synth.quant_matrix(fmt, m, k, seed=193, tensor_id=1, d_range=D_RANGE[fmt])
    q = rng.integers(-128, 128, (n, k))
    d = rng.uniform(1e-3, 0.5, (n, k // 32)).astype(np.float32)
    b = _blocks(q, d)
    wf = oracle.dequantize_f32(fmt, w, m, k).astype(np.float64).reshape(m, k)
    xf = (q.reshape(n, -1, 32) * d.astype(np.float64)[..., None]).reshape(n, k)
    ref = xf @ wf.T
    s = np.abs(xf) @ (np.abs(wf) + (np.abs(wf).max() if fmt in ("q4_1", "q5_1") else 0)).T
    for w_off, x_off, ldx, ldy in ((0, 0, None, None), (2, 4, 33 * 36 + 4, 50), (2, 0, 2000, 45)):
        y = _x8q(fmt, w, m, k, b, ldx, ldy, w_off, x_off)
        assert_within(y, ref, s, (k // 32 + 8) * U, f"x8q {fmt} {w_off} {ldx}")


@pytest.mark.parametrize("fmt", ["q8_0", "q4_1"])
@pytest.mark.parametrize("nb,n", [(9, 8), (10, 2), (131, 5)])
def test_x8q_infinite_scale_is_an_infinite_output(fmt, nb, n):
    """One block of one column with an infinite scale: that column's outputs
    are infinite with the sign of the block's product, the others as ever.
    The block is the last of the row, which a pass of four leaves short."""
    m, k = 37, 32 * nb
    rng = np.random.default_rng(nb)
    w = synth.quant_matrix(fmt, m, k, seed=195, tensor_id=nb, d_range=D_RANGE[fmt])
    q = rng.integers(-127, 128, (n, k))
    d = rng.uniform(0.1, 0.5, (n, nb)).astype(np.float32)
    if fmt == "q4_1":
        q[1, -32:] = 0                      # (its minimum would meet the scale too)
        q[1, -32] = 1
    d[1, -1] = np.inf
    wf = oracle.dequantize_f32(fmt, w, m, k).astype(np.float64).reshape(m, k)
    block = (q[1, -32:] * wf[:, -32:]).sum(-1)
    y = _x8q(fmt, w, m, k, _blocks(q, d))
    assert np.isfinite(np.delete(y, 1, 0)).all()
    if fmt == "q8_0":
        sure = np.abs(block) > 0
        assert np.array_equal(y[1][sure], np.sign(block[sure]) * np.inf)
    else:
        assert not np.isfinite(y[1]).any()


def test_x8q_nan_scale_and_empty_rows():
    m, k = 20, 128
    w = synth.quant_matrix("q4_0", m, k, seed=9, tensor_id=1, d_range=D_RANGE["q4_0"])
    d = np.ones((2, 4), np.float32)
    d[0, 2] = np.nan
    y = _x8q("q4_0", w, m, k, _blocks(np.ones((2, k)), d))
    assert np.isnan(y[0]).all() and np.isfinite(y[1]).all()
    t = torch()
    z = Guarded(2 * 5 * 4)
    dummy = t.zeros(64, dtype=t.uint8, device="cuda")
    assert qk.qk_mul_mat_vec_x8q("q4_1", dummy.data_ptr(), 5, 0, dummy.data_ptr(), 2, 0, z.ptr, 5, _stream()) == qk.QK_OK
    assert not z.host(np.float32).any() and z.guards_intact()
