"""GPU: qk_kv_store and qk_attn_decode through the C ABI and the binding.

The store is compared exactly with its rule in fp32 (numpy's conversions and
divisions round as the kernel's do).  The attention is compared with softmax
attention in 64 bits over the values that the cache holds.  Its tolerance, per
output, with A = sum_t p_t |V_t| / sum_t p_t and Z = the largest over t of
scale * log2(e) * sum_i |q_i K_ti| (both in 64 bits) and u = 2^-24:
  a score in log2: q as two parts (2^-21 of the row's largest |q|, so scale *
  log2(e) * 2^-21 * max|q| * sum|K| beside 2^-21 Z), D products summed in fp32
  (D u Z), four more roundings (4 u Z);
  so p is within ln2 times that, plus 2^-22 (exponential, scales) and 2^-21
  (two parts); numerator and denominator: twice, and T sums (T u each).
  Below fp32's range nothing is held: a probability under 2^-126 may count as
  0, which is 2^-126 sum_t |V_t| absolutely.
"""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import Guarded, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _say(*a):
    print("[case]", *a, flush=True)


class Pages:
    """A cache with known values: k, v in 64 bits per (sequence, head, token),
    laid out in pages in shuffled order; what no sequence holds is NaN (fp16)
    or a NaN scale with codes 127 (8 bits)."""

    def __init__(self, kind, lens, heads, dim, page, seed, room=None, tokens_outside_heads=False, spread=1.0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.kind, self.lens, self.heads, self.dim, self.page = kind, lens, heads, dim, page
        per = max(1, -(-(room or max(max(lens), 1)) // page))
        n_pages = len(lens) * per + 3
        self.table = rng.permutation(n_pages)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
        shape = (n_pages, heads, page, dim)
        pools = {}
        for p in "kv":
            x = (rng.standard_normal(shape) * spread).astype(np.float16)
            if kind == "f16":
                pools[p], sc = x, None
                val = x.astype(np.float64)
            else:
                c = np.clip(np.rint(x.astype(np.float32) * 40 / spread), -127, 127).astype(np.int8)
                # scales over several powers of two
                sc = (np.exp2(rng.uniform(-8, -2, shape[:3])) * spread).astype(np.float32)
                pools[p] = c
                val = c.astype(np.float64) * sc.astype(np.float64)[..., None]
            used = np.zeros((n_pages, page), bool)
            for s, n in enumerate(lens):
                for i in range(max(n, 0)):
                    used[self.table[s, i // page], i % page] = True
            free = ~used[:, None, :].repeat(heads, 1)
            if kind == "f16":
                pools[p][free] = np.nan
            else:
                pools[p][free] = 127
                sc[free] = np.nan
            pools[p + "s"] = sc
            setattr(self, p, [np.stack([val[self.table[s, i // page], :, i % page] for i in range(max(n, 0))], 1)
                              if n > 0 else np.zeros((heads, 0, dim)) for s, n in enumerate(lens)])

        def dev(a):
            if a is None:
                return None
            x = t.from_numpy(a).cuda()
            if tokens_outside_heads:
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            return x
        self.cache = qk.KVCache(dev(pools["k"]), dev(pools["v"]), dev(pools["ks"]), dev(pools["vs"]))
        self.dtable = t.from_numpy(self.table).cuda()
        self.dlens = t.from_numpy(np.asarray(lens, np.int32)).cuda()


def _reference(pg, q, scale, window, sinks):
    """(y, tolerance) in 64 bits."""
    n, hq, dim = q.shape
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(n):
        length = pg.lens[s]
        if length <= 0:
            continue
        t = np.arange(length)
        seen = (t >= length - window) | (t < sinks) if window else t >= 0
        for h in range(hq):
            K, V = pg.k[s][h * pg.heads // hq][seen], pg.v[s][h * pg.heads // hq][seen]
            x = q[s, h].astype(np.float64)
            z = K @ x * scale
            p = np.exp(z - z.max())
            y[s, h] = p @ V / p.sum()
            A = p @ np.abs(V) / p.sum()
            c = abs(scale) * 1.4426950408889634
            zz = (np.abs(K) @ np.abs(x)).max() * c
            zq = np.abs(K).sum(-1).max() * np.abs(x).max() * c
            dz = 2.0 ** -21 * (zz + zq) + (dim + 4) * U * zz
            tol[s, h] = (2 * (np.log(2) * dz + 2.0 ** -22 + 2.0 ** -21) + 2 * seen.sum() * U + 8 * U) * A + 2.0 ** -126 * np.abs(V).sum(0)
    return y, tol


def _attn(pg, q, scale=None, window=0, sinks=0, out="f32", max_len=None, offset=0):
    """y through the C ABI with guard bands."""
    t = torch()
    n, hq, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    room = pg.table.shape[1] * pg.page
    max_len = room if max_len is None else max_len
    qd = t.from_numpy(q.copy()).cuda()
    es = 4 if out == "f32" else 2
    y = Guarded(n * hq * dim * es, offset * es)
    need = qk.qk_attn_decode_workspace(pg.cache.desc, n, hq, max_len, window, sinks)
    ws = Guarded(need) if need else None
    st = qk.qk_attn_decode(pg.cache.desc, qd.data_ptr(), hq * dim, dim, n, hq, pg.dtable.data_ptr(),
                           pg.dtable.stride(0), pg.dlens.data_ptr(), max_len, scale, window, sinks,
                           qk.QK_F32 if out == "f32" else qk.QK_F16, y.ptr, hq * dim, dim, ws.ptr if ws else None, need,
                           t.cuda.current_stream().cuda_stream)
    assert st == qk.QK_OK, qk.status_string(st)
    got = y.host(np.float32 if out == "f32" else np.float16).reshape(n, hq, dim)
    assert y.guards_intact() and (ws is None or ws.guards_intact())
    return got


def _check(pg, q, got, scale=None, window=0, sinks=0, out="f32"):
    y, tol = _reference(pg, q, q.shape[2] ** -0.5 if scale is None else scale, window, sinks)
    if out == "f16":
        tol = tol + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
    err = np.abs(got.astype(np.float64) - y)
    assert np.all(err <= tol), f"worst {np.nanmax(err / np.maximum(tol, 1e-300))} of the tolerance"


def _q(n, hq, dim, seed, scale=1.5):
    return (np.random.default_rng(seed).standard_normal((n, hq, dim)) * scale).astype(np.float32)


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("page", [16, 24])
def test_attn_head_sizes(kind, dim, page):
    _say("attn", kind, dim, page)
    pg = Pages(kind, [1, 0, 31, 32, 33, 257, 700], 2, dim, page, dim + page)
    for group in (1, 5):
        q = _q(7, 2 * group, dim, dim)
        _check(pg, q, _attn(pg, q))


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("heads,hq", [(1, 1), (8, 8), (3, 12), (1, 16), (2, 34), (1, 71)])
def test_attn_head_groups(kind, heads, hq):
    _say("attn groups", kind, heads, hq)
    pg = Pages(kind, [130, 64, 7], heads, 64, 32, hq)
    q = _q(3, hq, 64, hq)
    _check(pg, q, _attn(pg, q))


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("page", [1, 7, 8, 16, 48, 100, 128])
def test_attn_page_sizes_and_layouts(kind, page):
    """Pages that end inside a tile; heads inside tokens; fp16 outputs."""
    _say("attn pages", kind, page)
    pg = Pages(kind, [page, page + 1, 3 * page - 1, 400], 2, 64, page, page, tokens_outside_heads=True)
    q = _q(4, 6, 64, page)
    _check(pg, q, _attn(pg, q, out="f16", offset=1), out="f16")


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (32, 0), (33, 4), (64, 32), (100, 33), (37, 50),
                                          (500, 4), (10, 300), (1000, 1000)])
def test_attn_window_and_sinks(kind, page, window, sinks):
    """Tokens that are not seen hold NaN, and table entries of pages without
    a token that is seen hold ids that are no pages: neither is used."""
    _say("attn window", kind, page, window, sinks)
    lens = [1, 2, 16, 33, 95, 128, 331, 600]
    pg = Pages(kind, lens, 2, 64, page, 7 * window + sinks)
    t = torch()
    table = pg.table.copy()
    pools = [pg.cache.k, pg.cache.v] if kind == "f16" else [pg.cache.k_scale, pg.cache.v_scale]
    for s, n in enumerate(lens):
        seen = np.zeros(table.shape[1] * page, bool)
        seen[max(0, n - window):n] = True
        seen[:min(sinks, n)] = True
        for i in np.flatnonzero(~seen[:n]):
            for x in pools:
                x[int(table[s, i // page]), :, int(i % page)] = float("nan")
        for p in range(table.shape[1]):
            if not seen[p * page:(p + 1) * page].any():
                table[s, p] = [-1, 2 ** 31 - 1, 10 ** 6][p % 3]
    pg.dtable = t.from_numpy(table).cuda()
    q = _q(len(lens), 4, 64, window)
    _check(pg, q, _attn(pg, q, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("lens", [[5000], [20011], [1, 9000, 4096, 0, 77]])
def test_attn_long_sequences_are_split_and_joined(kind, lens):
    _say("attn long", kind, lens)
    pg = Pages(kind, lens, 1, 64, 64, sum(lens))
    assert qk.qk_attn_decode_workspace(pg.cache.desc, len(lens), 4, max(lens)) > 0
    q = _q(len(lens), 4, 64, 3)
    a = _attn(pg, q)
    _check(pg, q, a)
    assert np.array_equal(a.view(np.uint32), _attn(pg, q).view(np.uint32)), "another run gave other bits"
    # another bound on the lengths: another split, within the tolerance
    _check(pg, q, _attn(pg, q, max_len=max(lens)))


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_attn_score_ranges(kind):
    """One token that takes all; equal scores; large and tiny queries; a zero
    query is the mean; a scale given by the caller."""
    pg = Pages(kind, [300, 300, 300, 300, 300], 1, 64, 16, 5)
    q = _q(5, 2, 64, 9)
    q[0] *= 40
    q[1] = 0
    q[2] *= 1e-20
    q[3] *= np.exp2(np.random.default_rng(1).uniform(-20, 3, q[3].shape))
    _check(pg, q, _attn(pg, q))
    _check(pg, q, _attn(pg, q, scale=-0.3), scale=-0.3)
    y = _attn(pg, q)
    mean = pg.v[1][0].mean(0)
    assert np.all(np.abs(y[1] - mean) <= (300 * U * 2 + 2.0 ** -19) * np.abs(pg.v[1][0]).mean(0))


def test_attn_many_small_probabilities_count():
    """100000 tokens at 2^-30 of the largest: together 1e-4 of the sum."""
    pg = Pages("f16", [100000], 1, 32, 128, 3)
    t = torch()
    k = pg.cache.k
    k.zero_()
    pg.cache.v.fill_(1.0)
    first = int(pg.table[0, 0])
    k[first, 0, 0, 0] = 1.0
    pg.cache.v[first, 0, 0] = 0.0
    q = np.zeros((1, 1, 32), np.float32)
    q[0, 0, 0] = 30 * np.log(2)
    y = _attn(pg, q, scale=1.0)
    p = 2.0 ** -30
    want = 99999 * p / (1 + 99999 * p)
    t.cuda.synchronize()
    # (a relative error of p, and of the sums of equal terms, T u)
    assert np.all(np.abs(y - want) <= want * (40 * np.log(2) * 2.0 ** -21 + 2.0 ** -19 + 1e5 * U * 2))


def test_attn_8_bit_scales_of_any_size():
    """Value scales from 2^-60 to 2^60 in one sequence, zero scales among them."""
    pg = Pages("i8", [640, 64], 1, 64, 16, 8)
    t = torch()
    rng = np.random.default_rng(2)
    for s, n in enumerate(pg.lens):
        e = np.exp2(rng.integers(-60, 61, n)).astype(np.float32)
        e[::7] = 0
        if s == 1:
            e[:] = 0
        c = pg.v[s][0]
        for i in range(n):
            page, slot = int(pg.table[s, i // 16]), i % 16
            old = float(pg.cache.v_scale[page, 0, slot])
            c[i] = np.rint(c[i] / old) * float(e[i])
            pg.cache.v_scale[page, 0, slot] = float(e[i])
    t.cuda.synchronize()
    q = _q(2, 3, 64, 4)
    _check(pg, q, _attn(pg, q))


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("page", [16, 12])
def test_attn_lengths_and_pages_out_of_range(kind, page):
    """Lengths of zero and below: zeros.  A length above max_len, a page id
    outside the pool: NaN for that sequence, the others as ever."""
    t = torch()
    pg = Pages(kind, [50, 50, 50, 50, 300], 2, 64, page, 6, room=320)
    q = _q(5, 4, 64, 2)
    want = _attn(pg, q)
    pg.dlens = t.tensor([0, -5, 301, 50, 300], dtype=t.int32, device="cuda")
    table = pg.table.copy()
    table[4, 200 // page] = pg.cache.n_pages
    pg.dtable = t.from_numpy(table).cuda()
    got = _attn(pg, q, max_len=300)
    assert not got[:2].any() and np.isnan(got[2]).all() and np.isnan(got[4]).all()
    pg.lens = [0, 0, 0, 50, 0]
    _check(pg, q, np.where(np.arange(5)[:, None, None] == 3, got, 0))
    assert np.allclose(got[3], want[3], rtol=1e-4, atol=1e-6)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_attn_non_finite_values_stay_in_their_row(kind):
    t = torch()
    pg = Pages(kind, [60, 60, 60], 2, 64, 16, 11)
    q = _q(3, 4, 64, 2)
    q[0, 1, 5] = np.inf
    q[0, 2, 5] = np.nan
    page = int(pg.table[1, 1])
    if kind == "f16":
        pg.cache.v[page, 1, 3, 7] = float("inf")
    else:
        pg.cache.v_scale[page, 1, 3] = float("inf")
    t.cuda.synchronize()
    y = _attn(pg, q)
    assert np.isnan(y[0, 1:3]).all() and np.isfinite(y[0, [0, 3]]).all()
    assert np.isfinite(y[1, :2]).all() and not np.isfinite(y[1, 2:, 7]).any()
    assert np.isfinite(y[2]).all()


def test_attn_strided_queries_and_outputs_another_stream_and_graph():
    t = torch()
    pg = Pages("f16", [90, 1500], 2, 64, 16, 12)
    q = _q(2, 4, 64, 2)
    want = _attn(pg, q)
    wide = t.full((2, 4, 80), float("nan"), device="cuda")
    wide[..., 8:72] = t.from_numpy(q).cuda()
    qd = wide[..., 8:72]
    y = t.full((4, 2, 64), 7.0, device="cuda").transpose(0, 1)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    qk.attn_decode(pg.cache, qd, pg.dtable, pg.dlens, y=y, stream=s)
    s.synchronize()
    assert np.array_equal(y.cpu().numpy(), want)
    out = t.empty(2, 4, 64, device="cuda")
    ws = qk.attn_decode_workspace(pg.cache, 2, 4, pg.dtable.shape[1] * 16)
    g = t.cuda.CUDAGraph()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        with t.cuda.graph(g, stream=s):
            qk.attn_decode(pg.cache, qd, pg.dtable, pg.dlens, y=out, workspace=ws)
    t.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(255)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want)


def test_attn_and_store_past_32_bit_offsets():
    """Pools of more than 2^32 bytes (2^31 elements): the last pages."""
    t = torch()
    n_pages, heads, page, dim = 2 ** 31 // (2 * 16 * 128) + 40, 2, 16, 128
    cache = qk.KVCache(*[t.empty((n_pages, heads, page, dim), dtype=t.float16, device="cuda") for _ in range(2)])
    pages = t.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=t.int32, device="cuda")
    rng = np.random.default_rng(3)
    k, v = (rng.standard_normal((40, heads, dim)).astype(np.float16).astype(np.float32) for _ in range(2))
    pos = t.arange(40, dtype=t.int32, device="cuda")
    qk.kv_store(cache, t.from_numpy(k).cuda(), t.from_numpy(v).cuda(), pages, pos,
                seq=t.zeros(40, dtype=t.int32, device="cuda"))
    assert np.array_equal(cache.k[n_pages - 1, :, 3].float().cpu().numpy(), k[3])
    q = _q(1, 4, dim, 5)
    y = qk.attn_decode(cache, t.from_numpy(q).cuda(), pages, t.tensor([40], dtype=t.int32, device="cuda")).cpu().numpy()

    class P:
        pass
    p = P()
    p.lens, p.heads = [40], heads
    p.k, p.v = [k.astype(np.float64).transpose(1, 0, 2)], [v.astype(np.float64).transpose(1, 0, 2)]
    _check(p, q, y)


def _store_ref(x, kind):
    x = x.astype(np.float32)
    if kind == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16), None
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        d = np.where(bad, np.float32(np.nan), top / np.float32(127)).astype(np.float32)
        q = np.clip(np.rint(x / d[..., None]), -127, 127)
    q = np.where((d > 0)[..., None], q, 0)
    return q.astype(np.int8), d


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim,heads,page,tokens", [(32, 1, 1, 1), (64, 3, 16, 37), (96, 2, 7, 50), (128, 8, 16, 64),
                                                   (160, 1, 5, 9), (256, 2, 32, 300), (224, 5, 24, 33)])
def test_store_matches_its_rule(kind, dim, heads, page, tokens):
    """Every byte of the pools: the new rows by the rule, the others untouched;
    tokens with no place (bad sequence, position or page) left out."""
    _say("store", kind, dim, heads, page, tokens)
    t = torch()
    rng = np.random.default_rng(dim + tokens)
    seqs, per = 4, -(-tokens // page)
    n_pages = seqs * per + 2
    table = rng.permutation(n_pages)[:seqs * per].reshape(seqs, per).astype(np.int32)
    # places drawn without repetition
    place = rng.permutation(seqs * per * page)[:tokens]
    seq, pos = (place // (per * page)).astype(np.int32), (place % (per * page)).astype(np.int32)
    k, v = (rng.standard_normal((tokens, heads, dim)).astype(np.float32) * np.exp2(rng.integers(-10, 10, (tokens, heads, 1))).astype(np.float32)
            for _ in range(2))
    k[0, 0] = 0
    v[-1, -1] = 1e-44
    k[-1, -1, 3] = np.inf
    v[0, 0, 1] = np.nan
    k[tokens // 2, 0] = 1e6                       # past fp16
    if tokens > 8:
        seq[1], pos[2], seq[3], pos[4] = seqs, -1, -1, per * page
        table[0, 0] = -1
        table[3, per - 1] = n_pages
    shape = (n_pages, heads, page, dim)
    nhd = dim % 64 == 0                           # heads inside tokens
    pools = []
    for _ in range(2):
        p = t.full((n_pages, page, heads, dim) if nhd else shape, 77, dtype=t.float16 if kind == "f16" else t.int8, device="cuda")
        pools.append(p.transpose(1, 2) if nhd else p)
    scales = [t.full((n_pages, page, heads), -1.0, device="cuda").transpose(1, 2) for _ in range(2)] if kind == "i8" else [None, None]
    cache = qk.KVCache(*pools, *scales)
    # strided inputs: k and v side by side
    kv = t.from_numpy(np.concatenate([k, v], 1)).cuda()
    qk.kv_store(cache, kv[:, :heads], kv[:, heads:], t.from_numpy(table).cuda(), t.from_numpy(pos).cuda(),
                seq=t.from_numpy(seq).cuda())
    t.cuda.synchronize()
    for x, pool, scale in ((k, pools[0], scales[0]), (v, pools[1], scales[1])):
        want = np.full(shape, 77, np.float16 if kind == "f16" else np.int8)
        wsc = np.full(shape[:3], -1.0, np.float32)
        c, d = _store_ref(x, kind)
        for i in range(tokens):
            if 0 <= seq[i] < seqs and 0 <= pos[i] < per * page and 0 <= table[seq[i], pos[i] // page] < n_pages:
                want[table[seq[i], pos[i] // page], :, pos[i] % page] = c[i]
                if kind == "i8":
                    wsc[table[seq[i], pos[i] // page], :, pos[i] % page] = d[i]
        assert np.array_equal(pool.cpu().numpy(), want, equal_nan=kind == "f16")
        if kind == "i8":
            assert np.array_equal(scale.cpu().numpy(), wsc, equal_nan=True)


def test_store_without_seq_then_attend():
    """A decode step's order: store the new token, attend with it."""
    t = torch()
    cache = qk.KVCache.empty(12, 2, 16, 64, "i8")
    table = t.arange(12, dtype=t.int32, device="cuda").view(3, 4)
    rng = np.random.default_rng(0)
    ks, vs = (rng.standard_normal((20, 3, 2, 64)).astype(np.float32) for _ in range(2))
    for i in range(20):
        qk.kv_store(cache, t.from_numpy(ks[i]).cuda(), t.from_numpy(vs[i]).cuda(), table,
                    t.full((3,), i, dtype=t.int32, device="cuda"))
    q = _q(3, 4, 64, 1)
    y = qk.attn_decode(cache, t.from_numpy(q).cuda(), table, t.full((3,), 20, dtype=t.int32, device="cuda")).cpu().numpy()

    class P:
        pass
    p = P()
    p.lens, p.heads = [20] * 3, 2

    def held(x):
        c, d = _store_ref(x, "i8")
        return (c.astype(np.float64) * d.astype(np.float64)[..., None]).transpose(1, 2, 0, 3)
    p.k, p.v = held(ks), held(vs)
    _check(p, q, y)
