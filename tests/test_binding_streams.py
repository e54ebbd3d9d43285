"""Where a call's own scratch is allocated: on the stream that the call runs
on, with tensors that only say where they are and a library that only notes
its calls (CPU)."""
import contextlib

import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from test_binding_places import Placed

F16, F32, I32 = torch.float16, torch.float32, torch.int32


class Scratch(Placed):
    nbytes = 1 << 20

    def __init__(self, pointer):
        super().__init__(0, torch.uint8, 1 << 20)
        self.pointer = pointer

    def data_ptr(self):
        return self.pointer


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 1 << 20
        return lambda *a: self.calls.append((name, a)) or 0


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def lib(monkeypatch):
    """The current stream is 64; `lib.scratch` lists the streams that scratch was allocated on, as the pointers given."""
    lib = Library()
    lib.scratch, current = [], [64]

    @contextlib.contextmanager
    def stream(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def empty(*a, **kw):
        lib.scratch.append(current[-1])
        return Scratch(1024 * current[-1] + 256)

    monkeypatch.setattr(pa, "load_library", lambda *a: lib)
    monkeypatch.setattr(pa, "_current_device", lambda: 0)
    monkeypatch.setattr(pa, "_current_stream", lambda device: 64)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch, "empty", empty)
    return lib


def t(dtype, *shape):
    return Placed(0, dtype, *shape)


def calls(**kw):
    """Every call that may allocate its own scratch."""
    k, v, table, lens = t(F16, 8, 2, 16, 64), t(F16, 8, 2, 16, 64), t(I32, 3, 4), t(I32, 3)
    q, w = t(F16, 3, 4, 64), t(F32, 3, 2, 64)
    w.size = lambda d: w.shape[d]
    table.size = lambda d: table.shape[d]
    lens.size = lambda d: lens.shape[d]
    cache = t(F16, 8, 16, 576)
    return dict(
        pa_decode=lambda: pa.pa_decode(q, q, k, v, table, lens, 64, 0.1, **kw),
        pa_decode_weights=lambda: pa.pa_decode_weights(q, w, q, k, v, table, lens, 64, 0.1, **kw),
        pa_evict_tokens=lambda: pa.pa_evict_tokens(k, v, table, lens, w, table, lens, w, 32, 4, **kw),
        pa_latent_decode=lambda: pa.pa_latent_decode(t(F16, 3, 4, 512), t(F16, 3, 4, 576), cache, table, lens, 64, 0.1,
                                                     **kw),
        pa_latent_prefill=lambda: pa.pa_latent_prefill(t(F16, 9, 2, 128), t(F16, 9, 2, 192), t(I32, 4),
                                                       t(F16, 2, 256, 512), cache, table, lens, 3, 64, 0.1, **kw))


CALLS = ["pa_decode", "pa_decode_weights", "pa_evict_tokens", "pa_latent_decode", "pa_latent_prefill"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("given,on", [(None, 64), (Stream(64), 64), (64, 64), (Stream(4096), 4096), (4096, 4096), (0, 0),
                                      (1, 0)])
def test_scratch_is_allocated_on_the_stream_of_the_call(lib, call, given, on):
    calls(stream=given)[call]()
    assert [name for name, _ in lib.calls] == [call]
    args = lib.calls[0][1]
    assert args[-1] == (64 if given is None else given if isinstance(given, int) else given.cuda_stream)
    assert lib.scratch == [on] and 1024 * on + 256 in args


@pytest.mark.parametrize("call", CALLS)
def test_a_given_workspace_is_taken_as_it_is(lib, call):
    calls(stream=4096, workspace=Scratch(1 << 30))[call]()
    assert lib.scratch == [] and 1 << 30 in lib.calls[0][1]


@pytest.mark.parametrize("call", CALLS)
def test_the_per_thread_stream_takes_a_given_workspace_only(lib, call):
    with pytest.raises(ValueError, match="needs a workspace"):
        calls(stream=2)[call]()
    calls(stream=2, workspace=Scratch(1 << 30))[call]()
    assert [name for name, _ in lib.calls] == [call]
