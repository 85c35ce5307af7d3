"""GPU: qk_attn_decode_shared where the first sequences of a group have ended,
in the order in which the calls on pages are used: a prompt is forked, its
sequences grow, some are dropped or cut short by kv_fork, whose table has -1
behind their tokens.  The others are answered as ever.

Tolerance of tests/test_gpu_attn_shared.py, whose reference in 64 bits and
whose arithmetic for it these tests take.
"""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch
from tests.test_gpu_attn_shared import U, Batch, _say

pytestmark = pytest.mark.gpu


class Forked(Batch):
    """groups: (sequences, prompt tokens); lens after the last step follow from
    `ended`: sequence -> tokens that it is cut to (0: dropped)."""

    def __init__(self, kind, groups, ended, heads=2, group=2, dim=64, page=16, seed=0):
        t = torch()
        rng = np.random.default_rng([seed, dim, page, len(ended)])
        self.kind, self.heads, self.group, self.dim, self.page = kind, heads, group, dim, page
        sizes, self.shared = [g[0] for g in groups], [g[1] for g in groups]
        self.starts = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        n = self.starts[-1]
        of = [g for g, s in enumerate(sizes) for _ in range(s)]
        own = rng.integers(1, 50, n)
        most = max(self.shared) + 60
        per = -(-most // page)
        n_pages = sum(-(-s // page) for s in self.shared) + n * (60 // page + 3)
        i32 = lambda x: t.tensor(np.asarray(x), dtype=t.int32, device="cuda")
        # the prompts, in pages of no order
        ids = iter(rng.permutation(n_pages).tolist())
        table = np.full((len(groups), per), -1, np.int32)
        for g, s in enumerate(self.shared):
            for j in range(-(-s // page)):
                table[g, j] = next(ids)
        first = [self.shared[g] + int(o) for g, o in zip(of, own)]
        t1, src, dst, missing = qk.kv_fork(i32(table), i32(self.shared), i32(first), page, n_pages, parent=i32(of))
        assert int(missing) == 0
        shape = (n_pages, heads, page, dim)
        self.cache = qk.KVCache.empty(*shape, dtype=kind)
        gen = t.Generator(device="cuda")
        gen.manual_seed(seed)
        for p in "kv":
            x = getattr(self.cache, p)
            if kind == "f16":
                x.normal_(generator=gen)
            else:
                x.random_(-127, 128, generator=gen)
                s = getattr(self.cache, p + "_scale")
                s.uniform_(0.005, 0.03, generator=gen)
        qk.kv_copy(self.cache, src, dst)
        # the next step, in which sequences end
        self.lens = [ended.get(s, n + 1) for s, n in enumerate(first)]
        t2, src, dst, missing = qk.kv_fork(t1, i32(first), i32(self.lens), page, n_pages)
        assert int(missing) == 0
        qk.kv_copy(self.cache, src, dst)
        self.dtable, self.dlens, self.dstarts, self.dshared = t2, i32(self.lens), i32(self.starts), i32(self.shared)
        self.table = t2.cpu().numpy()
        for s in ended:
            assert (self.table[s, -(-ended[s] // page):] == -1).all()
        self.at = [np.array([(self.table[s, i // page], i % page) for i in range(n)], np.int64).reshape(-1, 2)
                   for s, n in enumerate(self.lens)]
        self.val = {}
        for p in "kv":
            x = getattr(self.cache, p).double()
            if kind == "i8":
                x = x * getattr(self.cache, p + "_scale").double()[..., None]
            self.val[p] = x.cpu().numpy()
        self.max_len, self.max_shared, self.max_own = most, max(self.shared), 60
        self.of, self.ended, self.n_pages = of, ended, n_pages
        self.q = (rng.standard_normal((n, heads * group, dim)) * 1.5).astype(np.float32)

    def check(self, **kw):
        got = self.run(**kw)
        want, tol = self.reference()
        tol = tol + (np.abs(want) + tol) * U
        for s, n in enumerate(self.lens):
            if n <= 0:
                assert np.all(got[s] == 0), s
            elif n < self.shared[self.of[s]]:
                assert np.all(np.isnan(got[s])), s   # (it no longer has what its group shares)
            else:
                bad = ~(np.abs(got[s] - want[s]) <= tol[s])
                assert not bad.any(), (s, got[s][bad][:5], want[s][bad][:5], tol[s][bad][:5])
        return got


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("prompt", [1, 16, 40, 64, 129, 700])
@pytest.mark.parametrize("size", [2, 5, 20, 40])
def test_the_first_sequence_ends(kind, prompt, size):
    _say("first", kind, prompt, size)
    Forked(kind, [(size, prompt)], {0: 0}, seed=1).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
@pytest.mark.parametrize("dim,page", [(32, 8), (64, 7), (96, 16), (128, 16), (128, 24), (192, 16), (256, 32)])
def test_head_sizes_and_pages(kind, dim, page):
    """Rows by the tile of every size, in several chunks."""
    _say("dims", kind, dim, page)
    for size, group in ((2, 2), (9, 4), (40, 4)):
        Forked(kind, [(size, 1100)], {0: 0, 1: 0} if size > 2 else {0: 0}, 1, group, dim, page, seed=2).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_cut_short(kind):
    """First sequences that keep a part of what their group shares, within a
    page and to its end; and whole groups that have ended."""
    for cut in ({0: 1}, {0: 16}, {0: 100}, {0: 0, 1: 17, 2: 299}, {0: 33, 3: 0, 6: 0}):
        _say("cut", kind, cut)
        Forked(kind, [(7, 300)], cut, seed=3).check()
    _say("all ended", kind)
    Forked(kind, [(3, 300), (4, 70), (2, 50)], {0: 0, 1: 0, 2: 0, 3: 0, 7: 0}, seed=4).check()
    # more than a wave's lanes of them before the first that goes on
    for n in (63, 64, 65, 140):
        _say("many ended", kind, n)
        Forked(kind, [(3, 40), (150, 90), (2, 33)], {3 + s: s % 2 * 20 for s in range(n)}, 1, 1, seed=5).check()


@pytest.mark.parametrize("kind", ["f16", "i8"])
def test_no_other_result_changes(kind):
    """A sequence's result is the same bits whether or not others of its group
    have ended; a bad page that is everybody's still is refused."""
    t = torch()
    b = Forked(kind, [(6, 200), (20, 333)], {}, seed=6)
    ref = b.check()
    for gone in ([0], [6], [0, 1, 2, 6, 7], [5, 25]):
        table, lens = b.dtable.clone(), b.dlens.clone()
        b.dtable[gone] = -1
        b.dlens[gone] = 0
        got = b.run()
        want = ref.copy()
        want[gone] = 0
        assert np.array_equal(got, want), gone
        # what an ended row holds of its pages is followed, as before it ended
        b.dtable.copy_(table)
        assert np.array_equal(b.run(), want), gone
        b.dlens.copy_(lens)
    b.dtable[0], b.dlens[0] = -1, 0
    b.dtable[1, 1] = -1
    got = b.run()
    assert np.all(got[0] == 0) and np.all(np.isnan(got[1:6])) and np.array_equal(got[6:], ref[6:])


def test_replayed_graph():
    """One captured call, before and after the first sequences end."""
    t = torch()
    b = Forked("f16", [(6, 200), (20, 333)], {}, seed=7)
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
    for gone in (None, 0, 6, 1, 7):
        if gone is not None:
            b.dtable[gone], b.dlens[gone] = -1, 0
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(got, call()) and not t.isnan(got).any(), gone
