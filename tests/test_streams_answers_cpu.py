"""The stream of the calls on pages, shared attention and log probabilities,
and the memory that they make for themselves, as tests/test_streams_cpu.py has
it for the others; no GPU is touched."""
import pytest
import torch

from dequant_quantized_gemv_amd import qk
from tests.test_streams_cpu import HERE, THERE, Stub, record  # noqa: F401


def _calls():
    table, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = qk.KVCache(*[torch.zeros(8, 2, 16, 64, dtype=torch.float16) for _ in range(2)])
    q, x = torch.zeros(2, 4, 64), torch.zeros(2, 64)
    starts = torch.zeros(2, dtype=torch.int32)
    return {
        "fork": lambda s: qk.kv_fork(table, n, n, 16, 8, stream=s),
        "compact": lambda s: qk.kv_compact(table, n, 16, 8, stream=s),
        "shared": lambda s: qk.attn_decode_shared(cache, q, table, n, starts, starts[:1], stream=s),
        "logprobs": lambda s: qk.token_logprobs(x, n, top=2, stream=s),
        "copy": lambda s: qk.kv_copy(cache, n, n, stream=s),
    }


@pytest.mark.parametrize("call", ["fork", "compact", "shared", "logprobs", "copy"])
@pytest.mark.parametrize("handle", [THERE, HERE, 0, None])
@pytest.mark.parametrize("as_object", [False, True])
def test_memory_comes_from_the_stream_that_runs(record, call, handle, as_object):  # noqa: F811
    fn = _calls()[call]
    record.made.clear()
    fn(Stub(handle) if as_object and handle is not None else handle)
    want = HERE if handle is None else handle
    assert record.ran == [want]
    assert (call == "copy") == (not record.made) and set(record.made) <= {want}
    assert record.current == HERE
