"""GPU: qk_kv_fork, qk_kv_compact and qk_kv_copy against their rules taken one
row and one page after another: every id, move and byte must be equal."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import Guarded, torch

pytestmark = pytest.mark.gpu


def _say(*a):
    print("[case]", *a, flush=True)


def fork_reference(table, lens, new_lens, page, n_pages, parent, out_pages):
    rows, per = table.shape
    parent = range(len(new_lens)) if parent is None else parent
    plan, held = [], {}
    for p, n in zip(parent, new_lens):
        had = min(max(int(lens[p]), 0), per * page) if 0 <= p < rows else 0
        has = min(max(int(n), 0), out_pages * page)
        row = [int(x) for x in table[p][:-(-min(had, has) // page)]] if had else []
        for x in row:
            if 0 <= x < n_pages:
                held[x] = held.get(x, 0) + 1
        plan.append((row, had, has))
    free = [x for x in range(n_pages) if x not in held][::-1]
    out = np.full((len(plan), out_pages), -1, np.int32)
    src, dst = np.full(len(plan), -1, np.int32), np.full(len(plan), -1, np.int32)
    missing = 0
    for i, (row, had, has) in enumerate(plan):
        if has > had and had % page and held.get(row[had // page], 0) > 1:
            if free:
                src[i], dst[i] = row[had // page], free[-1]
            else:
                missing += 1
            row[had // page] = free.pop() if free else -1
        while len(row) < -(-has // page):
            missing += not free
            row.append(free.pop() if free else -1)
        out[i, :len(row)] = row
    return out, src, dst, missing


def compact_reference(table, lens, page, n_pages):
    rows, per = table.shape
    kept = [[int(x) for x in r[:-(-min(max(int(n), 0), per * page) // page)]] for r, n in zip(table, lens)]
    live = sorted({x for r in kept for x in r if 0 <= x < n_pages})
    src = [x for x in live if x >= len(live)]
    there = set(live)
    dst = [x for x in range(len(live)) if x not in there]
    to = dict(zip(src, dst))
    out = np.full((rows, per), -1, np.int32)
    for o, r in zip(out, kept):
        o[:len(r)] = [to.get(x, x) for x in r]
    pad = [-1] * (n_pages // 2 - len(src))
    return out, np.array(src + pad, np.int32), np.array(dst + pad, np.int32), len(live)


def _table(rng, rows, per, n_pages, how):
    """Ids of a table: distinct pages, pages met several times, or those with
    ids outside the pool among them."""
    if how == "distinct":
        return rng.permutation(max(n_pages, rows * per))[:rows * per].reshape(rows, per).astype(np.int32)
    t = rng.integers(0, n_pages, (rows, per)).astype(np.int32)
    if how == "bad":
        t[rng.random((rows, per)) < 0.1] = rng.choice([-1, n_pages, 2 ** 31 - 1, -2 ** 31])
    return t


def _dev(a, pad=0):
    """A tensor of the rows of `a`, each followed by `pad` other elements."""
    t = torch()
    a = np.ascontiguousarray(a, dtype=np.int32)
    if a.ndim == 1 or not pad:
        return t.from_numpy(a.copy()).cuda()
    wide = np.full((a.shape[0], a.shape[1] + pad), 12345, np.int32)
    wide[:, :a.shape[1]] = a
    return t.from_numpy(wide).cuda()[:, :a.shape[1]]


FORKS = [  # rows, pages in, new rows, pages out, page size, pool
    (1, 1, 1, 1, 1, 1), (1, 4, 8, 4, 16, 20), (4, 63, 4, 63, 16, 300), (3, 5, 7, 9, 24, 64), (2, 3, 5, 0, 16, 33),
    (64, 256, 64, 256, 16, 17000), (300, 7, 1100, 8, 1, 9000), (5, 40, 1025, 41, 100, 40000), (7, 100, 9, 100, 8, 400000),
    (2, 33000, 3, 33001, 1, 100000), (0, 0, 3, 4, 16, 40), (3, 0, 3, 4, 16, 5),
]


@pytest.mark.parametrize("shape", FORKS, ids=str)
@pytest.mark.parametrize("how", ["distinct", "again", "bad"])
@pytest.mark.parametrize("parents", ["none", "one", "any"])
def test_fork(shape, how, parents):
    rows, per, n, out_pages, page, n_pages = shape
    _say("fork", shape, how, parents)
    rng = np.random.default_rng([rows, per, n, page, len(how), len(parents)])
    table = _table(rng, rows, per, n_pages, how)
    lens = rng.integers(-3, per * page + 4, rows).astype(np.int32)
    parent = None if parents == "none" else np.full(n, rows // 2, np.int32) if parents == "one" else \
        rng.integers(-2, rows + 2, n).astype(np.int32)
    at = np.arange(n) if parent is None else parent
    old = np.array([lens[p] if 0 <= p < rows else 0 for p in at], np.int64)
    new = np.clip(old + rng.integers(-2 * page, 2 * page + 2, n), -5, out_pages * page + 5)
    some = rng.random(n) < 0.2
    new[some] = rng.integers(0, out_pages * page + 1, n)[some]
    if rows:
        # (lengths at the ends of pages too)
        new[rng.random(n) < 0.2] = min(page, out_pages * page)
    want = fork_reference(table, lens, new, page, n_pages, parent, out_pages)
    need = qk.qk_kv_pages_workspace(n, n_pages)
    ws, out = Guarded(need, fill=0xA5), Guarded(4 * n * (out_pages + 3))
    src, dst, missing = Guarded(4 * n), Guarded(4 * n), Guarded(4)
    dt, dl, dn = _dev(table, 2), _dev(lens), _dev(new)
    dp = _dev(parent) if parent is not None else None
    for _ in range(2):  # (the second call finds the scratch as the first left it)
        st = qk.qk_kv_fork(dt.data_ptr(), dt.stride(0) if rows > 1 else per, dl.data_ptr(), rows, per,
                           dp.data_ptr() if dp is not None else None, dn.data_ptr(), n, out_pages, page, n_pages, out.ptr,
                           out_pages + 3, src.ptr, dst.ptr, missing.ptr, ws.ptr, need)
        assert st == qk.QK_OK
        got = out.host(np.int32).reshape(n, out_pages + 3)
        ld = out_pages + 3
        assert np.array_equal(got[:, :out_pages], want[0])
        if n > 1:
            assert np.all(got[:, out_pages:].reshape(-1).view(np.uint8) == 0xA5), (ld, "past the rows")
        assert np.array_equal(src.host(np.int32), want[1]) and np.array_equal(dst.host(np.int32), want[2])
        assert missing.host(np.int32)[0] == want[3]
        assert all(g.guards_intact() for g in (ws, out, src, dst, missing))


@pytest.mark.parametrize("shape", [(4, 63, 16, 300), (64, 256, 16, 17000), (5, 40, 100, 400000)], ids=str)
def test_fork_in_place(shape):
    rows, per, page, n_pages = shape
    _say("fork in place", shape)
    t = torch()
    rng = np.random.default_rng(5)
    table = _table(rng, rows, per, n_pages, "again")
    lens = rng.integers(0, per * page + 1, rows).astype(np.int32)
    new = np.minimum(lens + rng.integers(0, 3, rows), per * page).astype(np.int32)
    want = fork_reference(table, lens, new, page, n_pages, None, per)
    dt = _dev(table, 3)
    out, src, dst, missing = qk.kv_fork(dt, _dev(lens), _dev(new), page, n_pages, out=dt)
    assert out is dt
    for got, w in zip((dt, src, dst), want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert missing.item() == want[3]
    # packed in place as well
    want = compact_reference(want[0], new, page, n_pages)
    out, src, dst, live = qk.kv_compact(dt, _dev(new), page, n_pages, out=dt)
    for got, w in zip((dt, src, dst), want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert live.item() == want[3]
    t.cuda.synchronize()


COMPACTS = [  # rows, pages, page size, pool
    (1, 1, 1, 1), (1, 1, 16, 2), (4, 63, 16, 300), (3, 5, 24, 15), (64, 512, 16, 65536), (300, 7, 1, 9000), (1100, 5, 8, 33000),
    (7, 100, 8, 400000), (2, 33000, 1, 100000), (0, 0, 16, 40), (3, 0, 16, 5), (6, 16, 16, 97),
]


@pytest.mark.parametrize("shape", COMPACTS, ids=str)
@pytest.mark.parametrize("how", ["distinct", "again", "bad", "high", "all"])
def test_compact(shape, how):
    rows, per, page, n_pages = shape
    _say("compact", shape, how)
    rng = np.random.default_rng([rows, per, page, len(how)])
    if how == "high":      # everything has to move
        table = (n_pages - 1 - np.arange(rows * per) % max(1, n_pages // 2)).reshape(rows, per).astype(np.int32)
    elif how == "all":     # nothing has to
        table = (np.arange(rows * per) % n_pages).reshape(rows, per).astype(np.int32)
    else:
        table = _table(rng, rows, per, n_pages, how)
    lens = rng.integers(-3, per * page + 4, rows).astype(np.int32)
    if how == "all":
        lens[:] = per * page
    want = compact_reference(table, lens, page, n_pages)
    need = qk.qk_kv_pages_workspace(rows, n_pages)
    moves = n_pages // 2
    ws, out = Guarded(need), Guarded(4 * rows * (per + 1))
    src, dst, live = Guarded(4 * moves), Guarded(4 * moves), Guarded(4)
    dt, dl = _dev(table, 2), _dev(lens)
    for _ in range(2):
        st = qk.qk_kv_compact(dt.data_ptr(), per + 2, dl.data_ptr(), rows, per, page, n_pages, out.ptr, per + 1, src.ptr, dst.ptr,
                              live.ptr, ws.ptr, need) if rows != 1 else \
            qk.qk_kv_compact(dt.data_ptr(), per, dl.data_ptr(), rows, per, page, n_pages, out.ptr, per, src.ptr, dst.ptr, live.ptr,
                             ws.ptr, need)
        assert st == qk.QK_OK
        got = out.host(np.int32)
        got = got.reshape(rows, per + 1)[:, :per] if rows != 1 else got[:per].reshape(1, per)
        assert np.array_equal(got, want[0])
        assert np.array_equal(src.host(np.int32), want[1]) and np.array_equal(dst.host(np.int32), want[2])
        assert live.host(np.int32)[0] == want[3]
        assert all(g.guards_intact() for g in (ws, out, src, dst, live))


def _pools(rng, kind, order, heads, page, dim, n_pages, gap):
    """Keys, values (and scales) of random bytes as views (page, head, slot, ...)
    of tensors whose dimensions lie in the given order ("k": keys and values in
    one tensor), `gap` unused rows behind each innermost step."""
    t = torch()
    size = {"p": n_pages, "k": 2, "h": heads, "s": page}

    def make(row, dtype, high):
        shape = [size[d] for d in order]
        shape[-1] += gap
        whole = t.from_numpy(rng.integers(0, high, shape + row).astype(dtype)).cuda()
        if whole.dtype == t.int16:
            whole = whole.view(t.float16)
        cut = whole.narrow(len(shape) - 1, 0, size[order[-1]])
        if "k" not in order:
            return [cut.permute([order.index(d) for d in "phs"] + [3] * bool(row))]
        at, rest = order.index("k"), [d for d in order if d != "k"]
        return [cut.select(at, i).permute([rest.index(d) for d in "phs"] + [3] * bool(row)) for i in range(2)]
    row, dtype, high = ([dim], np.int16, 2 ** 15) if kind == "f16" else ([dim], np.int8, 127)
    kv = make(row, dtype, high)
    kv = kv if len(kv) == 2 else kv + make(row, dtype, high)
    if kind == "i8":
        sc = make([], np.float32, 1000)
        kv += sc if len(sc) == 2 else sc + make([], np.float32, 1000)
    return kv


def _bits(x):
    t = torch()
    return x.contiguous().view({2: t.int16, 1: t.int8, 4: t.int32}[x.element_size()])


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("order,gap", [("phs", 0), ("psh", 0), ("hps", 0), ("phs", 3), ("psh", 1), ("sph", 0), ("pkhs", 0), ("pskh", 0), ("phsk", 0)])
@pytest.mark.parametrize("dims", [(3, 16, 64, 21), (1, 1, 32, 40), (8, 24, 128, 12), (2, 100, 96, 9), (1, 7, 256, 5), (5, 1, 160, 11)], ids=str)
def test_copy(kind, order, gap, dims):
    heads, page, dim, n_pages = dims
    _say("copy", kind, order, gap, dims)
    t = torch()
    rng = np.random.default_rng([heads, page, dim, gap, len(order)])
    kv = _pools(rng, kind, order, heads, page, dim, n_pages, gap)
    cache = qk.KVCache(*kv)
    before = [x.clone() for x in kv]
    ids = rng.permutation(n_pages)
    n = n_pages // 2
    src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
    src[0], dst[-1] = -1, n_pages
    if n > 2:
        src[1] = src[2]      # one page to two places
    qk.kv_copy(cache, _dev(src), _dev(dst))
    for x, b in zip(kv, before):
        for a, c in zip(src, dst):
            if 0 <= a < n_pages and 0 <= c < n_pages:
                b[int(c)] = b[int(a)]
        assert t.equal(_bits(x), _bits(b))


def test_copy_leaves_what_lies_between():
    """Elements between the rows and pages of a cache stay as they are."""
    t = torch()
    whole = t.arange(2 * 6 * 40 * 48, dtype=t.int32, device="cuda").to(t.int16).view(t.float16).view(2, 6, 40, 48)
    before = whole.clone()
    # 2 heads of 16 slots of 32 in pages of 40 rows of 48
    kv = [whole[i].as_strided((6, 2, 16, 32), (1920, 768, 48, 1), whole[i].storage_offset()) for i in range(2)]
    cache = qk.KVCache(*kv)
    qk.kv_copy(cache, _dev([1, 4]), _dev([3, 0]))
    for i in range(2):
        want = before[i].as_strided((6, 2, 16, 32), (1920, 768, 48, 1), before[i].storage_offset())
        want[3], want[0] = want[1].clone(), want[4].clone()
    assert t.equal(whole.view(t.int16), before.view(t.int16))


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_many_large_and_many_small_pages(kind):
    """More than the caches hold (other stores), and small pages of which a
    workgroup takes several, pairs left out among them."""
    t = torch()
    for pairs, heads, page, dim in ((1200, 8, 16, 128), (3000, 1, 8, 32), (700, 2, 3, 32)):
        n = 2 * pairs + 3
        g = t.Generator(device="cuda")
        g.manual_seed(pairs)
        cache = qk.KVCache.empty(n, heads, page, dim, kind)
        for x in (cache.k, cache.v):
            x.random_(-127, 128, generator=g) if kind == "i8" else x.normal_(generator=g)
        if kind == "i8":
            cache.k_scale.normal_(generator=g)
            cache.v_scale.normal_(generator=g)
        ids = t.randperm(n, device="cuda", generator=g).to(t.int32)
        src, dst = ids[:pairs].clone(), ids[pairs:2 * pairs].clone()
        src[5], dst[9], src[17] = -1, n, dst[17]
        ok = t.ones(pairs, dtype=t.bool, device="cuda")
        ok[5] = ok[9] = False
        want = []
        for x in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            if x is not None:
                w = x.clone()
                w[dst[ok].long()] = x[src[ok].long()]
                want.append((x, w))
        qk.kv_copy(cache, src, dst)
        for x, w in want:
            assert t.equal(_bits(x), _bits(w)), (pairs, kind)


def test_same_page_and_no_pairs():
    t = torch()
    cache = qk.KVCache.empty(4, 2, 16, 64)
    cache.k.normal_()
    was = cache.k.clone()
    qk.kv_copy(cache, _dev([2, 2]), _dev([2, 1]))
    was[1] = was[2]
    assert t.equal(cache.k, was)
    qk.kv_copy(cache, _dev(np.zeros(0)), _dev(np.zeros(0)))
    assert t.equal(cache.k, was)


def test_plans_in_a_graph():
    """fork, copy and compact captured once and replayed over changing tables,
    eager work between the replays."""
    t = torch()
    rng = np.random.default_rng(3)
    rows, per, page, n_pages = 9, 40, 16, 500
    cache = qk.KVCache.empty(n_pages, 2, page, 64, "i8")
    table, lens, new, parent = (t.zeros(s, dtype=t.int32, device="cuda") for s in ((rows, per), rows, rows, rows))
    ws = [qk.kv_pages_workspace(rows, n_pages) for _ in range(2)]

    def step():
        f = qk.kv_fork(table, lens, new, page, n_pages, parent=parent, workspace=ws[0])
        qk.kv_copy(cache, f[1], f[2])
        c = qk.kv_compact(f[0], new, page, n_pages, workspace=ws[1])
        qk.kv_copy(cache, c[1], c[2])
        return f + c

    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        step()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=s):
            got = step()
    t.cuda.current_stream().wait_stream(s)
    for i in range(5):
        tb = _table(rng, rows, per, n_pages, "again")
        ln = rng.integers(0, per * page + 1, rows).astype(np.int32)
        pa = rng.integers(0, rows, rows).astype(np.int32)
        nw = np.minimum(ln[pa] + rng.integers(0, 40, rows), per * page).astype(np.int32)
        for d, h in ((table, tb), (lens, ln), (new, nw), (parent, pa)):
            d.copy_(t.from_numpy(h))
        cache.k.random_(-127, 127)
        cache.k_scale.normal_()
        k, ks = cache.k.clone(), cache.k_scale.clone()
        graph.replay()
        t.cuda.synchronize()
        f = fork_reference(tb, ln, nw, page, n_pages, pa, per)
        c = compact_reference(f[0], nw, page, n_pages)
        for a, b in zip(got, f + c):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), i
        for a, b in [(f[1], f[2]), (c[1], c[2])]:
            for x, y in zip(a, b):
                if x >= 0:
                    k[int(y)], ks[int(y)] = k[int(x)], ks[int(x)]
        assert t.equal(cache.k, k) and t.equal(cache.k_scale, ks)
