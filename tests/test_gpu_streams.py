"""GPU: a call on another stream than the current one takes its outputs and its
scratch from that stream's pool (the allocator's own record of its segments
says whose a block is), and gives the values that it gives on the current one."""
import numpy as np
import pytest

from dequant_quantized_gemv_amd import qk, synth
from tests.gpu_helpers import D_RANGE, torch

pytestmark = pytest.mark.gpu


def _pool(ptr):
    """Handle of the stream whose pool holds the address."""
    for s in torch().cuda.memory_snapshot():
        if s["address"] <= ptr < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError(f"no segment holds {ptr:#x}")


def _calls():
    t = torch()
    g = np.random.default_rng(1)
    x = t.from_numpy(g.standard_normal((2, 64)).astype(np.float32)).cuda()
    w = t.from_numpy(synth.quant_matrix("q4_0", 96, 64, seed=5, tensor_id=1, d_range=D_RANGE["q4_0"])).cuda()
    xh, x8 = x.half(), qk.rms_norm(x, out_dtype="x8")
    cache = qk.KVCache(*[t.from_numpy(g.standard_normal((256, 2, 16, 64)).astype(np.float16)).cuda() for _ in range(2)])
    table = t.arange(256, dtype=t.int32, device="cuda").view(2, 128)
    q = t.from_numpy(g.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
    lens = t.tensor([2000, 700], dtype=t.int32, device="cuda")
    ids = t.tensor([[0, 2], [1, 1]], dtype=t.int32, device="cuda")
    return {
        "dequantize": lambda **k: [qk.dequantize("q4_0", w, 96, 64, **k)],
        "gemv": lambda **k: [qk.mul_mat_vec("q4_0", w, 96, 64, x, **k)],
        "gemv x8": lambda **k: [qk.mul_mat_vec_x8("q4_0", w, 96, 64, x, **k)],
        "batched": lambda **k: qk.mul_mat_vec_batched("q4_0", [(w, 96, 64, x), (w, 32, 64, x)], **k),
        "id": lambda **k: [qk.mul_mat_vec_id("q4_0", w, 3, 32, 64, ids, x, **k)],
        "gemm": lambda **k: [qk.mul_mat("q4_0", w, 96, 64, xh, **k)],
        "norm": lambda **k: qk.rms_norm(x, residual=x, **k),
        "norm x8": lambda **k: [qk.rms_norm(x, out_dtype="x8", **k)],
        "x8q": lambda **k: [qk.mul_mat_vec_x8q("q4_0", w, 96, 64, x8, **k)],
        "attn": lambda **k: [qk.attn_decode(cache, q, table, lens, **k)],
        "route": lambda **k: qk.moe_route(x, 4, **k),
    }


@pytest.mark.parametrize("name", ["dequantize", "gemv", "gemv x8", "batched", "id", "gemm", "norm", "norm x8", "x8q", "attn", "route"])
def test_outputs_and_scratch_are_of_the_stream_that_runs(name, monkeypatch):
    t = torch()
    call = _calls()[name]
    want = call()
    scratch = []
    if name == "attn":
        lib, ran = qk.load(), qk.load().qk_attn_decode

        class Seen:
            def __getattr__(self, f):
                return getattr(lib, f)

            def qk_attn_decode(self, *a):
                scratch.append(a[-3])
                return ran(*a)
        monkeypatch.setattr(qk, "load", lambda: Seen())
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = call(stream=stream)
        s.synchronize()
        for a, b in zip(want, got):
            assert t.equal(a, b) and _pool(b.data_ptr()) == s.cuda_stream
    assert len(scratch) == (2 if name == "attn" else 0)
    for ptr in scratch:
        assert ptr is not None and _pool(ptr) == s.cuda_stream
    # the null stream, while another one is current
    with t.cuda.stream(s):
        got = call(stream=0)
        t.cuda.default_stream().synchronize()
        for a, b in zip(want, got):
            assert t.equal(a, b) and _pool(b.data_ptr()) == 0
