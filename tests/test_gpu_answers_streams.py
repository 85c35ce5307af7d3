"""GPU: the calls on pages, shared attention and log probabilities on another
stream than the current one take their outputs and scratch from that
stream's pool and give the same values."""
import pytest

from dequant_quantized_gemv_amd import qk
from tests.gpu_helpers import torch
from tests.test_gpu_streams import _pool

pytestmark = pytest.mark.gpu


def _calls():
    t = torch()
    cache = qk.KVCache.empty(64, 2, 16, 64)
    cache.k.normal_()
    cache.v.normal_()
    table = t.arange(64, dtype=t.int32, device="cuda").view(4, 16)
    lens = t.tensor([100, 90, 17, 200], dtype=t.int32, device="cuda")
    starts, shared = (t.tensor(x, dtype=t.int32, device="cuda") for x in ([0, 2, 4], [32, 16]))
    q = t.randn(4, 4, 64, device="cuda")
    x = t.randn(3, 70000, device="cuda")
    ids = t.zeros(3, 2, dtype=t.int32, device="cuda")
    return {
        "fork": lambda **k: qk.kv_fork(table, lens, lens + 1, 16, 64, **k),
        "compact": lambda **k: qk.kv_compact(table, lens, 16, 64, **k),
        "attn": lambda **k: [qk.attn_decode_shared(cache, q, table, lens, starts, shared, **k)],
        "logprobs": lambda **k: qk.token_logprobs(x, ids, top=3, **k),
    }


@pytest.mark.parametrize("name", ["fork", "compact", "attn", "logprobs"])
def test_outputs_and_scratch_are_of_the_stream_that_runs(name, monkeypatch):
    t = torch()
    call = _calls()[name]
    want = call()
    scratch = []
    lib = qk.load()

    class Seen:
        def __getattr__(self, f):
            fn = getattr(lib, f)
            if f.endswith("workspace"):
                return fn

            def ran(*a):
                scratch.append(a[-3])
                return fn(*a)
            return ran
    monkeypatch.setattr(qk, "load", lambda: Seen())
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = call(stream=stream)
        s.synchronize()
        for a, b in zip(want, got):
            assert t.equal(a, b) and _pool(b.data_ptr()) == s.cuda_stream
    assert len(scratch) == 2
    for ptr in scratch:
        assert ptr is not None and _pool(ptr) == s.cuda_stream
    with t.cuda.stream(s):
        got = call(stream=0)
        t.cuda.default_stream().synchronize()
        for a, b in zip(want, got):
            assert t.equal(a, b) and _pool(b.data_ptr()) == 0


def test_copy_on_another_stream():
    t = torch()
    cache = qk.KVCache.empty(6, 2, 16, 64)
    cache.k.normal_()
    src, dst = (t.tensor(x, dtype=t.int32, device="cuda") for x in ([0, 1], [4, 5]))
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    for stream in (s, s.cuda_stream, 0, None):
        cache.k[4:] = 0
        t.cuda.synchronize()
        qk.kv_copy(cache, src, dst, stream=stream)
        t.cuda.synchronize()
        assert t.equal(cache.k[4:], cache.k[:2])
