"""The stream of a call and the memory that the call makes for itself: outputs
and scratch must come from the pool of the stream that the work runs on, for a
block of another stream's pool may still be in use there.  The library and
torch's stream calls are replaced by records of what they were asked; no GPU
is touched."""
import contextlib

import pytest
import torch

from dequant_quantized_gemv_amd import qk

HERE, THERE = 0x1000, 0x2000


class Stub:
    """A stream: its handle."""

    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Record:
    """The current stream, and for each allocation and launch the stream that
    it was made for."""

    def __init__(self):
        self.current, self.made, self.ran = HERE, [], []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace"):
                return 4096
            handle = args[-1]
            self.ran.append(handle)
            return qk.QK_OK
        return call


@pytest.fixture
def record(monkeypatch):
    r = Record()
    t = torch.cuda

    @contextlib.contextmanager
    def stream(s):
        before, r.current = r.current, s.cuda_stream
        yield
        r.current = before

    def kept(fn):
        def make(*args, **kw):
            r.made.append(r.current)
            kw.pop("device", None)
            return fn(*args, **kw)
        return make
    monkeypatch.setattr(qk, "load", lambda: r)
    monkeypatch.setattr(qk, "_same_device", lambda *ts: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: r.current, raising=False)
    monkeypatch.setattr(t, "current_stream", lambda device=None: Stub(r.current))
    monkeypatch.setattr(t, "default_stream", lambda device=None: Stub(0))
    monkeypatch.setattr(t, "ExternalStream", Stub)
    monkeypatch.setattr(t, "stream", stream)
    f, i = torch.zeros(2, 64), torch.zeros(2, 4, dtype=torch.int32)
    cache = qk.KVCache(*[torch.zeros(8, 2, 16, 64, dtype=torch.float16) for _ in range(2)])
    w, x8 = torch.zeros(64 * 2 * 18, dtype=torch.uint8), torch.zeros(2, 72, dtype=torch.uint8)
    q, lens = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    r.calls = {
        "dequantize": lambda s: qk.dequantize("q4_0", w, 64, 64, stream=s),
        "gemv": lambda s: qk.mul_mat_vec("q4_0", w, 64, 64, f, stream=s),
        "gemv x8": lambda s: qk.mul_mat_vec_x8("q4_0", w, 64, 64, f, stream=s),
        "batched": lambda s: qk.mul_mat_vec_batched("q4_0", [(w, 64, 64, f), (w, 32, 64, f)], stream=s),
        "id": lambda s: qk.mul_mat_vec_id("q4_0", w, 2, 32, 64, i, f, stream=s),
        "gemm": lambda s: qk.mul_mat("q4_0", w, 64, 64, f.half(), stream=s),
        "norm": lambda s: qk.rms_norm(f, residual=f.clone(), stream=s),
        "norm x8": lambda s: qk.rms_norm(f, out_dtype="x8", stream=s),
        "x8q": lambda s: qk.mul_mat_vec_x8q("q4_0", w, 64, 64, x8, stream=s),
        "attn": lambda s: qk.attn_decode(cache, q, i, lens, stream=s),
        "attn y": lambda s: qk.attn_decode(cache, q, i, lens, y=q.clone(), stream=s),
        "route": lambda s: qk.moe_route(f, 4, stream=s),
    }
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, kept(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "new_empty", kept(torch.Tensor.new_empty))
    return r


@pytest.mark.parametrize("call", ["dequantize", "gemv", "gemv x8", "batched", "id", "gemm", "norm", "norm x8", "x8q", "attn",
                                  "attn y", "route"])
@pytest.mark.parametrize("handle", [THERE, HERE, 0, None])
@pytest.mark.parametrize("as_object", [False, True])
def test_memory_comes_from_the_stream_that_runs(record, call, handle, as_object):
    record.calls[call](Stub(handle) if as_object and handle is not None else handle)
    want = HERE if handle is None else handle
    assert record.ran == [want]
    assert record.made and set(record.made) == {want}
    assert record.current == HERE
