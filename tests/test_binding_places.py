"""Where the binding lets tensors lie, with tensors that only say where they
are and a library that only notes its calls (CPU)."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa


class Placed:
    """What the binding asks of a contiguous CUDA tensor."""

    def __init__(self, device, dtype, *shape):
        self.device, self.index, self.dtype, self.shape = f"cuda:{device}", device, dtype, torch.Size(shape)

    is_cuda = True

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "pa_decode_workspace_size":
            return lambda *a: 256
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(pa, "load_library", lambda *a: lib)
    monkeypatch.setattr(pa, "_current_device", lambda: 0)
    monkeypatch.setattr(pa, "_current_stream", lambda device: 0)
    return lib


def _calls(cache_dtype, device):
    """Every call with all of its tensors on the device."""
    t = lambda dtype, *shape: Placed(device, dtype, *shape)    # noqa: E731
    f16, i32, i64 = torch.float16, torch.int32, torch.int64
    shape = pa.fp4_cache_shape(4, 2, 16, 64) if cache_dtype == "fp4" else (4, 2, 16, 64)
    k, v, host = (t(f16 if cache_dtype == "f16" else torch.uint8, *shape) for _ in range(3))
    kw = dict(cache_dtype=cache_dtype)
    attend = (k, v, t(i32, 3, 4), t(i32, 3))
    rows = lambda: t(f16, 3, 4, 64)                            # noqa: E731
    return dict(
        pa_reshape_and_cache=lambda: pa.pa_reshape_and_cache(t(f16, 3, 2, 64), t(f16, 3, 2, 64), t(i64, 3), k, v, **kw),
        pa_decode=lambda: pa.pa_decode(rows(), rows(), *attend, 64, 0.1, workspace=t(torch.uint8, 256), **kw),
        pa_decode_static_scratch=lambda: pa.pa_decode_static_scratch(rows(), rows(), *attend, 64, 0.1, **kw),
        pa_prefill=lambda: pa.pa_prefill(rows(), rows(), t(i32, 4), *attend, 1, 0.1, **kw),
        pa_copy_blocks=lambda: pa.pa_copy_blocks(k, v, t(i64, 1, 2), **kw),
        pa_swap_blocks=lambda: pa.pa_swap_blocks(k, v, host, host, t(i64, 1, 2), "out", **kw),
        pa_gather_cache=lambda: pa.pa_gather_cache(t(f16, 3, 2, 64), t(f16, 3, 2, 64), t(i64, 3), k, v, **kw),
        pa_compact_blocks=lambda: pa.pa_compact_blocks(k, v, t(i64, 1, 2), t(i32, 3, 4), t(i32, 3), **kw))


OLDER = ["pa_reshape_and_cache", "pa_decode", "pa_decode_static_scratch", "pa_prefill", "pa_copy_blocks",
         "pa_swap_blocks"]
NEWER = ["pa_gather_cache", "pa_compact_blocks"]


@pytest.mark.parametrize("call", OLDER)
@pytest.mark.parametrize("cache_dtype", ["f16", "e4m3", "int8"])
@pytest.mark.parametrize("device", [0, 1])
def test_memory_that_the_current_device_may_reach_is_taken(lib, call, cache_dtype, device):
    """Tensors of another device reach the library, which launches on the
    current one: with access between the two they are as good as its own."""
    _calls(cache_dtype, device)[call]()
    assert lib.calls == [call]


@pytest.mark.parametrize("call", OLDER + NEWER)
@pytest.mark.parametrize("cache_dtype", ["f16", "int8", "fp4"])
def test_four_bit_caches_and_newer_calls_stay_on_the_current_device(lib, call, cache_dtype):
    _calls(cache_dtype, 0)[call]()
    assert lib.calls == [call]
    if cache_dtype == "fp4" or call in NEWER:
        with pytest.raises(ValueError, match="must be on the current device"):
            _calls(cache_dtype, 1)[call]()
        assert lib.calls == [call]


def test_a_type_given_as_a_number_object_is_read_at_every_call():
    """Codes held in arrays: not hashable, or changed between two calls."""
    import numpy as np
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    code = lambda x: pa._describe(k, x, 1.0, 1.0)[2]           # noqa: E731
    assert code("int8") == code(pa.PA_INT8) == code(np.int64(pa.PA_INT8)) == code(np.array(pa.PA_INT8)) == pa.PA_INT8
    t = torch.tensor(pa.PA_INT8)
    assert code(t) == pa.PA_INT8
    t.fill_(pa.PA_FP8_E4M3)
    assert code(t) == pa.PA_FP8_E4M3
