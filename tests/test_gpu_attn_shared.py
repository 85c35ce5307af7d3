"""GPU: qk_attn_decode_shared through the C ABI and the binding, against softmax
attention in 64 bits over the values that the cache holds.

Tolerance as of the decode attention (tests/test_gpu_attn.py), with A = sum_t p_t |V_t|
/ sum_t p_t, Z the largest over t of scale * log2(e) * sum_i |q_i K_ti|, u = 2^-24:
  scores: 2^-21 (Z + scale * log2(e) * max|q| * sum|K|) + (D + 4) u Z in log2, ln2 of
  which is relative in p; p itself 2^-22 (exponential, scales) and 2^-21 (its
  parts); numerator and denominator: twice, and T sums (T u each), 8 u to join.
  fp16 values meet p in parts that stop at 2^-36 of the largest p: 2^-36 sum_t |V_t|
  / sum_t p_t besides.
  Below fp32's range nothing is held: 2^-126 sum_t |V_t|.
"""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import Guarded, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ELSEWHERE = 2 ** 30  # a page id that must not be followed


def _say(*a):
    print("[case]", *a, flush=True)


class Batch:
    """groups: (sequences, shared tokens); own: tokens of its own of each
    sequence (None: lens <= 0).  What no token holds is NaN; entries of the
    pages that only shared tokens lie in are bad ids but in a group's first
    sequence."""

    def __init__(self, kind, groups, own, heads, group, dim, page, seed=0, lead=0, spread=1.0, layout="phs"):
        t = torch()
        rng = np.random.default_rng([seed, heads, dim, page, len(own)])
        self.kind, self.heads, self.group, self.dim, self.page = kind, heads, group, dim, page
        n = len(own)
        self.starts = [lead]
        for size, _ in groups:
            self.starts.append(self.starts[-1] + size)
        assert self.starts[-1] <= n
        self.shared = [s for _, s in groups]
        of = [-1] * n
        for g, (a, b) in enumerate(zip(self.starts, self.starts[1:])):
            of[a:b] = [g] * (b - a)
        self.of = of
        have = [max(self.shared[g], 0) if g >= 0 else 0 for g in of]
        self.lens = [-3 if o is None else h + o for h, o in zip(have, own)]
        self.max_len = max(max(self.lens), 1)
        per = -(-self.max_len // page)
        # pages: each sequence its own for its tokens; the first of a group for the shared ones too
        held = []
        for s in range(n):
            lo = 0 if of[s] < 0 or s == self.starts[of[s]] else have[s] // page
            hi = -(-max(self.lens[s], have[s] if of[s] >= 0 and s == self.starts[of[s]] else 0) // page)
            held.append((lo, max(lo, hi)))
        n_pages = sum(b - a for a, b in held) + 2
        ids = iter(rng.permutation(n_pages))
        self.table = np.full((n, per), ELSEWHERE, np.int32)
        for s, (a, b) in enumerate(held):
            self.table[s, a:b] = [next(ids) for _ in range(b - a)]
        shape = (n_pages, heads, page, dim)
        pools, val = {}, {}
        for p in "kv":
            x = (rng.standard_normal(shape) * spread).astype(np.float16)
            if kind == "f16":
                pools[p], sc, val[p] = x, None, x.astype(np.float64)
            else:
                c = np.clip(np.rint(x.astype(np.float32) * 40 / spread), -127, 127).astype(np.int8)
                sc = (np.exp2(rng.uniform(-8, -2, shape[:3])) * spread).astype(np.float32)
                pools[p], val[p] = c, c.astype(np.float64) * sc.astype(np.float64)[..., None]
            pools[p + "s"] = sc
        used = np.zeros((n_pages, page), bool)
        self.at = []
        for s in range(n):
            places = []
            for i in range(max(self.lens[s], 0)):
                row = self.starts[of[s]] if of[s] >= 0 and i < have[s] else s
                places.append((self.table[row, i // page], i % page))
            self.at.append(np.array(places, np.int64).reshape(-1, 2))
            used[self.at[s][:, 0], self.at[s][:, 1]] = True
        for g, a in enumerate(self.starts[:-1]):  # (shared tokens are there, whoever sees them)
            if a < self.starts[g + 1]:
                i = np.arange(max(self.shared[g], 0))
                used[self.table[a, i // page], i % page] = True
        free = ~used[:, None, :].repeat(heads, 1)
        for p in "kv":
            if kind == "f16":
                pools[p][free] = np.nan
            else:
                pools[p][free] = 127
                pools[p + "s"][free] = np.nan
        self.val, self.pools, self.n_pages = val, pools, n_pages

        def dev(a):
            if a is None:
                return None
            x = t.from_numpy(a).cuda()
            return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "psh" else x
        self.cache = qk.KVCache(dev(pools["k"]), dev(pools["v"]), dev(pools["ks"]), dev(pools["vs"]))
        i32 = lambda x: t.from_numpy(np.asarray(x, np.int32)).cuda()
        self.dtable, self.dlens, self.dstarts, self.dshared = i32(self.table), i32(self.lens), i32(self.starts), i32(self.shared)
        self.max_shared = max([0] + self.shared)
        self.max_own = max([1] + [o for o in own if o is not None])
        self.q = (rng.standard_normal((n, heads * group, dim)) * 1.5).astype(np.float32)

    def reference(self, scale=None):
        n, hq, dim = self.q.shape
        scale = dim ** -0.5 if scale is None else scale
        y, tol = np.zeros(self.q.shape), np.zeros(self.q.shape)
        c = abs(scale) * 1.4426950408889634
        for s in range(n):
            if self.lens[s] <= 0:
                continue
            pg, sl = self.at[s][:, 0], self.at[s][:, 1]
            for h in range(self.heads):
                K, V = (self.val[p][pg, h, sl] for p in "kv")
                rows = slice(h * self.group, (h + 1) * self.group)
                x = self.q[s, rows].astype(np.float64)
                z = x @ K.T * scale
                p = np.exp(z - z.max(-1, keepdims=True))
                total = p.sum(-1, keepdims=True)
                y[s, rows] = p @ V / total
                A = p @ np.abs(V) / total
                zz = (np.abs(x) @ np.abs(K).T).max(-1, keepdims=True) * c
                zq = np.abs(K).sum(-1).max() * np.abs(x).max(-1, keepdims=True) * c
                dz = 2.0 ** -21 * (zz + zq) + (dim + 4) * U * zz
                sv = np.abs(V).sum(0)
                tol[s, rows] = (2 * (np.log(2) * dz + 2.0 ** -22 + 2.0 ** -21) + 2 * len(K) * U + 8 * U) * A + 2.0 ** -126 * sv
                if self.kind == "f16":
                    tol[s, rows] += 2.0 ** -36 * sv / total
        return y, tol

    def run(self, scale=None, out="f32", bounds=None, fill=0xA5):
        """y through the C ABI with guard bands."""
        t = torch()
        n, hq, dim = self.q.shape
        scale = dim ** -0.5 if scale is None else scale
        max_len, max_shared, max_own = bounds or (self.max_len, self.max_shared, self.max_own)
        qd = t.from_numpy(self.q.copy()).cuda()
        es = 4 if out == "f32" else 2
        y = Guarded(n * hq * dim * es)
        need = qk.qk_attn_decode_shared_workspace(self.cache.desc, n, hq, max_len, max_shared, max_own)
        assert need > 0
        ws = Guarded(need, fill=fill)
        st = qk.qk_attn_decode_shared(self.cache.desc, qd.data_ptr(), hq * dim, dim, n, hq, self.dtable.data_ptr(),
                                      self.dtable.stride(0), self.dlens.data_ptr(), max_len, self.dstarts.data_ptr(),
                                      self.dshared.data_ptr(), len(self.shared), max_shared, max_own, scale,
                                      qk.QK_F32 if out == "f32" else qk.QK_F16, y.ptr, hq * dim, dim, ws.ptr, need)
        assert st == qk.QK_OK
        got = y.host(np.float32 if out == "f32" else np.float16).reshape(n, hq, dim).astype(np.float64)
        assert y.guards_intact() and (fill != 0xA5 or ws.guards_intact())
        return got

    def check(self, scale=None, out="f32", bounds=None):
        got = self.run(scale, out, bounds)
        want, tol = self.reference(scale)
        if out == "f16":
            tol = tol + (np.abs(want) + tol) * 2.0 ** -11 + 2.0 ** -25
        else:
            tol = tol + (np.abs(want) + tol) * U
        bad = ~(np.abs(got - want) <= tol)
        for s, n in enumerate(self.lens):
            if n <= 0:
                assert np.all(got[s] == 0), s
        assert not bad.any(), (np.argwhere(bad)[:5].tolist(), got[bad][:5], want[bad][:5], tol[bad][:5], int(bad.sum()))


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("size", [2, 20])
def test_head_sizes(kind, dim, size):
    """Few rows of a group (64 at a time) and many (128)."""
    _say("dim", kind, dim, size)
    rng = np.random.default_rng(dim)
    Batch(kind, [(size, 150)], rng.integers(0, 70, size).tolist(), 2, 4, dim, 16, seed=1).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("shared", [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_shared_lengths(kind, shared):
    _say("shared", kind, shared)
    for size, page in ((3, 16), (11, 24), (40, 7)):
        own = [1, 0 if shared else 1, 5, None, 31, 32, 33, 64, 2, 1, 100][:size] + [1] * max(0, size - 11)
        Batch(kind, [(size, shared)], own, 1, 3, 64, page, seed=2).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 48, 100, 1024])
@pytest.mark.parametrize("layout", ["phs", "psh"])
def test_pages(kind, page, layout):
    _say("page", kind, page, layout)
    Batch(kind, [(4, 333), (13, 200)], [17] * 17, 3, 2, 64, page, seed=3, layout=layout).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 16, 17, 71])
@pytest.mark.parametrize("size", [1, 6, 30])
def test_query_heads(kind, group, size):
    _say("group", kind, group, size)
    Batch(kind, [(size, 300)], [3 + i for i in range(size)], 2, group, 64, 16, seed=4).check()


GROUPS = [
    [(1, 70)] * 9, [(4, 0), (4, 100), (4, -5), (4, 64)], [(0, 50), (3, 129), (0, 0), (7, 1000), (1, 5), (0, 7)],
    [(2, 40 + i) for i in range(70)], [(1, i) for i in range(130)], [(50, 513)], [(90, 17), (1, 900), (33, 256)], [],
]


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("which", range(len(GROUPS)))
@pytest.mark.parametrize("lead,behind", [(0, 0), (3, 2)])
def test_groups(kind, which, lead, behind):
    """Groups of every size, empty ones, more than a wave's lanes of them, and
    sequences before and behind that belong to none."""
    groups = GROUPS[which]
    n = lead + sum(s for s, _ in groups) + behind
    if n == 0:
        return
    _say("groups", kind, which, lead, behind)
    rng = np.random.default_rng(which)
    own = [None if rng.random() < 0.1 else int(rng.integers(1, 60)) for _ in range(n)]
    Batch(kind, groups, own, 2, 3, 64, 16, seed=5, lead=lead).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("heads,group,dim,size,shared,own", [
    (8, 4, 128, 4, 9000, 40), (1, 8, 64, 3, 40000, 3000), (2, 4, 128, 24, 5000, 700), (1, 1, 32, 200, 3000, 10), (4, 16, 128, 9, 4100, 33),
    (1, 2, 256, 5, 7000, 100)])
def test_long(kind, heads, group, dim, size, shared, own):
    """Shared and own tokens in several parts."""
    _say("long", kind, heads, group, dim, size, shared, own)
    rng = np.random.default_rng(size)
    Batch(kind, [(size, shared)], rng.integers(1, own + 1, size).tolist(), heads, group, dim, 16, seed=6).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("heads,group,dim,page,n,layout", [
    (8, 1, 64, 24, 131, "phs"), (8, 4, 128, 16, 130, "phs"), (4, 17, 32, 16, 129, "psh"), (1, 2, 64, 7, 1025, "phs"),
    (1, 1, 96, 32, 1027, "phs"), (16, 1, 256, 16, 66, "phs")])
def test_many_sequences(kind, heads, group, dim, page, n, layout):
    """A wave takes a sequence's own tokens alone (not where they may be many)."""
    _say("many", kind, heads, group, dim, page, n, layout)
    rng = np.random.default_rng(n)
    own = [None if rng.random() < 0.05 else int(rng.choice([0, 1, 7, 32, 33, 65, 100])) for _ in range(n)]
    own[5], own[n - 1] = 480, 300
    groups = [(20, 150), (3, 40), (1, 129), (32, 65)]
    for s in range(2, 2 + sum(g[0] for g in groups)):
        own[s] = own[s] if own[s] != 0 or s % 2 else 1
    b = Batch(kind, groups, own, heads, group, dim, page, seed=11, lead=2, layout=layout)
    b.check()
    b.check(bounds=(b.max_len, b.max_shared, b.max_len))
    # a page outside the pool: its sequence alone is NaN
    y = b.run()
    at = b.lens[5] // b.page - 1
    b.dtable[5, at] = b.n_pages
    got = b.run()
    assert np.isnan(got[5]).all()
    got[5] = y[5]
    assert np.array_equal(got, y)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_half_outputs_scales_and_bounds(kind):
    b = Batch(kind, [(5, 260), (20, 90)], [9] * 25, 2, 4, 64, 16, seed=7)
    b.check(out="f16")
    b.check(scale=1.0)
    b.check(scale=-0.3)
    b.check(scale=0.0)
    first = b.run()
    # the same on every run, and whatever the scratch holds
    assert np.array_equal(first, b.run(fill=0)) and np.array_equal(first, b.run(fill=0xFF))
    room = b.table.shape[1] * b.page
    for bounds in ((room, b.max_shared, b.max_own), (room, room, b.max_own), (room, b.max_shared, room), (room, room, room)):
        b.check(bounds=bounds)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_large_and_small_values(kind):
    for spread in (1e-6 if kind == "i8" else 1e-3, 100.0):
        for mul in (1e-20, 1e-3, 30.0, 1e15):
            b = Batch(kind, [(3, 200), (30, 150)], [20] * 33, 1, 2, 64, 16, seed=8, spread=spread)
            b.q *= np.float32(mul)
            b.check(scale=0.125 if mul < 1 else 0.125 / mul)


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_refusals_on_the_device(kind):
    """Sequences that cannot be answered are NaN, the others as ever."""
    t = torch()
    groups, own = [(3, 100), (20, 70), (2, 30)], [5] * 25
    b = Batch(kind, groups, own, 2, 2, 64, 16, seed=9)
    ref = b.run()

    def expect(rows, **kw):
        got = b.run(**kw)
        for s in range(25):
            if s in rows:
                assert np.all(np.isnan(got[s])), s
            else:
                assert np.array_equal(got[s], ref[s]), s
    # a bad page among the shared ones: the group; of its own: the sequence
    for bad in (-1, b.n_pages, ELSEWHERE, -2 ** 31):
        keep = b.dtable.clone()
        b.dtable[0, 1] = bad
        b.dtable[5, 4] = bad
        expect({0, 1, 2, 5})
        b.dtable.copy_(keep)
    # shorter than what is shared; more tokens than any bound
    b.dlens[1] = 99
    b.dlens[24] = 10 ** 9
    expect({1, 24})
    b.dlens.copy_(t.tensor(b.lens, dtype=t.int32))
    # (other bounds may split otherwise: only the refused ones are looked at)
    got = b.run(bounds=(b.max_len, 99, b.max_own))
    assert np.all(np.isnan(got[:3])) and not np.any(np.isnan(got[3:]))
    got = b.run(bounds=(b.max_len, b.max_shared, 4))
    assert np.all(np.isnan(got))
    got = b.run(bounds=(104, b.max_shared, 100))
    assert np.all(np.isnan(got[:3])) and not np.any(np.isnan(got[3:]))
    # groups out of order or outside the batch
    for starts in ([0, 3, 2, 25], [-1, 3, 23, 25], [0, 3, 23, 26], [25, 0, 0, 0], [0, 2 ** 31 - 1, 3, 25], [0, -2 ** 31, 23, 25]):
        b.dstarts.copy_(t.tensor(starts, dtype=t.int32))
        assert np.all(np.isnan(b.run())), starts


def test_infinite_keys():
    """A key that overflowed fp16: probability 0 with a score of -infinity, NaN
    with +infinity or -infinity alone, with every size of the low part of q."""
    for size in (2, 20):
        b = Batch("f16", [(size, 96)], [7] * size, 1, 2, 32, 16, seed=10)
        k = b.pools["k"].copy()
        where = [(3, 5), (60, 9), (98, 0)]   # (token, dim), the last one of the first sequence's own
        for tok, d in where:
            page, slot = b.at[0][tok]
            k[page, 0, slot, d] = np.inf
        b.cache.k.copy_(torch().from_numpy(k))
        for exact in (False, True):
            b.q[:, 0] = -np.abs(b.q[:, 0])   # head 0: -infinity; head 1: +infinity
            b.q[:, 1] = np.abs(b.q[:, 1])
            if exact:
                b.q = b.q.astype(np.float16).astype(np.float32)
                b.q[:, :, 7] = 2.0           # (a low part of 0 in every dimension: powers of two)
                b.q = np.sign(b.q) * np.exp2(np.round(np.log2(np.abs(b.q) + 1e-3))).astype(np.float32)
            got = b.run(scale=1.0)
            for s in range(size):
                z = b.at[s]
                K, V = b.val["k"][z[:, 0], 0, z[:, 1]], b.val["v"][z[:, 0], 0, z[:, 1]]
                seen = np.ones(len(K), bool)
                seen[[3, 60] + ([98] if s == 0 else [])] = False
                x = b.q[s, 0].astype(np.float64)
                p = np.exp((K @ x) - (K[seen] @ x).max()) * seen
                assert np.allclose(got[s, 0], p @ V / p.sum(), atol=1e-4), (size, exact, s)
                assert np.all(np.isnan(got[s, 1])), (size, exact, s)


def test_strides_streams_and_binding():
    t = torch()
    b = Batch("f16", [(3, 90), (12, 140)], [11] * 15, 2, 4, 64, 16, seed=11)
    q = t.from_numpy(b.q).cuda()
    args = (b.cache, q, b.dtable, b.dlens, b.dstarts, b.dshared)
    kw = dict(max_len=b.max_len, max_shared=b.max_shared, max_own=b.max_own)
    ref = t.from_numpy(b.run()).float().cuda()
    assert t.equal(qk.attn_decode_shared(*args, **kw), ref)
    # heads outside sequences, rows with something between them
    qw = t.zeros(8, 15, 80, device="cuda")
    qv = qw[:, :, 8:72].transpose(0, 1)
    qv.copy_(q)
    yw = t.full((8, 15, 70), 7.0, device="cuda")
    yv = yw[:, :, :64].transpose(0, 1)
    tw = t.full((15, b.table.shape[1] + 3), 5, dtype=t.int32, device="cuda")
    tw[:, :-3] = b.dtable
    got = qk.attn_decode_shared(b.cache, qv, tw[:, :-3], *args[3:], y=yv, **kw)
    assert t.equal(got, ref) and t.all(yw[:, :, 64:] == 7.0)
    ws = qk.attn_decode_shared_workspace(b.cache, 40, 8, 4096, 2048, 500)
    assert t.equal(qk.attn_decode_shared(*args, workspace=ws, **kw), ref)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = qk.attn_decode_shared(*args, stream=s, **kw)
    s.synchronize()
    assert t.equal(got, ref)
    assert qk.attn_decode_shared(b.cache, q[:0], b.dtable[:0], b.dlens[:0], b.dstarts[:1], b.dshared[:0]).shape == (0, 8, 64)
    want = qk.attn_decode_shared(*args)   # default bounds
    assert t.allclose(want, ref, atol=1e-5, rtol=0)


def test_others_do_not_change_a_result():
    """What the sequences of other groups hold, and how long they are."""
    t = torch()
    b = Batch("f16", [(3, 90), (12, 140), (2, 33)], [11] * 17, 2, 4, 64, 16, seed=12)
    ref = b.run()
    b.dlens[3:15] = t.tensor([140 + i % 3 if i % 4 else 0 for i in range(12)], dtype=t.int32)
    b.dshared[1] = 120
    got = b.run()
    assert np.array_equal(got[:3], ref[:3]) and np.array_equal(got[15:], ref[15:])


def test_replayed_graph():
    t = torch()
    b = Batch("i8", [(3, 300), (12, 500)], [40] * 15, 2, 4, 64, 16, seed=13)
    q = t.from_numpy(b.q).cuda()
    call = lambda: qk.attn_decode_shared(b.cache, q, b.dtable, b.dlens, b.dstarts, b.dshared, max_len=b.max_len,
                                         max_shared=b.max_shared, max_own=b.max_own)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        call()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=s):
            got = call()
    t.cuda.current_stream().wait_stream(s)
    for i in range(4):
        q.normal_()
        b.dlens.copy_(t.tensor([300 + 10 * i + k for k in range(3)] + [500 + i + k for k in range(12)], dtype=t.int32))
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(got, call()), i


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_offsets_past_32_bits(kind):
    """Pages of more than 4 GiB of keys; a copy among them."""
    t = torch()
    heads, page, dim = 8, 64, 128
    one = heads * page * dim * (2 if kind == "f16" else 1)
    n_pages = (5 << 30) // one
    free, _ = t.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("not enough memory")
    cache = qk.KVCache.empty(n_pages, heads, page, dim, kind)
    at = [n_pages - 1, n_pages - 2, 3, n_pages - 5, n_pages - 7, 9]
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    for p in at[:4] + at[4:]:
        if kind == "f16":
            cache.k[p].normal_(generator=g)
            cache.v[p].normal_(generator=g)
        else:
            cache.k[p].random_(-127, 128, generator=g)
            cache.v[p].random_(-127, 128, generator=g)
            cache.k_scale[p].fill_(0.02)
            cache.v_scale[p].fill_(0.02)
    table = t.tensor([[at[0], at[1], at[2], at[3]], [-1, -1, at[4], at[5]]], dtype=t.int32, device="cuda")
    lens, starts, shared = (t.tensor(x, dtype=t.int32, device="cuda") for x in ([250, 200], [0, 2], [128]))
    q = t.randn(2, 32, dim, device="cuda", generator=g)
    y = qk.attn_decode_shared(cache, q, table, lens, starts, shared)
    # the same pages in a small cache
    small = qk.KVCache.empty(6, heads, page, dim, kind)
    for i, p in enumerate(at):
        for a, b in ((small.k, cache.k), (small.v, cache.v)) + (((small.k_scale, cache.k_scale), (small.v_scale, cache.v_scale)) if kind == "i8" else ()):
            a[i] = b[p]
    st = t.tensor([[0, 1, 2, 3], [-1, -1, 4, 5]], dtype=t.int32, device="cuda")
    assert t.equal(y, qk.attn_decode_shared(small, q, st, lens, starts, shared))
    qk.kv_copy(cache, t.tensor([at[0], 9], dtype=t.int32, device="cuda"), t.tensor([1, n_pages - 9], dtype=t.int32, device="cuda"))
    assert t.equal(cache.k[1], cache.k[at[0]]) and t.equal(cache.v[n_pages - 9], cache.v[9])
