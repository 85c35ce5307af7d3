"""The scratch that a call makes for itself lives until the library has taken
the call: before that its block must not go back to the pool, where another
thread could be given it.  The library is replaced by a record; no GPU is
touched."""
import weakref

import pytest
import torch

from dequant_quantized_gemv_amd import qk
from tests.test_streams_answers_cpu import _calls
from tests.test_streams_cpu import record  # noqa: F401


@pytest.mark.parametrize("call", ["fork", "compact", "shared", "logprobs", "attn"])
def test_scratch_lives_until_the_library_returns(record, monkeypatch, call):  # noqa: F811
    made, alive = [], []
    empty = torch.empty

    def make(*args, **kw):
        x = empty(*args, **kw)
        if x.dtype is torch.uint8:
            made.append((x.data_ptr(), weakref.ref(x)))
        return x

    class Library:
        def __getattr__(self, name):
            fn = getattr(record, name)

            def ran(*args):
                if not name.endswith("workspace"):
                    alive.extend(ref() is not None for ptr, ref in made if ptr in args)
                return fn(*args)
            return ran
    fn = _calls()[call] if call != "attn" else record.calls[call]
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(qk, "load", lambda: Library())
    fn(None)
    assert len(made) == 1 and alive == [True]
