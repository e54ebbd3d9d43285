"""A decode's workspace in memory that the call ahead of it on the stream still
reads, as an allocator hands out a tensor freed between the two calls.

Each call ahead reads one of its inputs to the end of a long run; the decode's
workspace is the end of that input.  Stream order is all the caller has to
keep: neither call may see the other's writes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from tests._fp4 import DEV, random_cache

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _write(cache_dtype, T=32768):
    """(input read to the end, call, outputs): rows of many prompts written."""
    H, D, bs = 8, 128, 16
    shape = pa.fp4_cache_shape(T // bs, H, bs, D) if cache_dtype == "fp4" else (T // bs, H, bs, D)
    caches = [torch.zeros(shape, dtype=torch.bfloat16 if cache_dtype == "bf16" else torch.uint8, device=DEV)
              for _ in range(2)]
    key, value = (torch.randn(T, H, D, generator=_gen(i), device=DEV).bfloat16() for i in range(2))
    slots = torch.randperm(T, generator=_gen(2), device=DEV)
    return key, lambda: pa.pa_reshape_and_cache(key, value, slots, *caches, cache_dtype=cache_dtype), caches


def _gather(cache_dtype):
    T, H, D, bs, nb = 1 << 19, 2, 64, 16, 4096
    rng = np.random.default_rng(3)
    if cache_dtype == "fp4":
        caches = [torch.from_numpy(random_cache(rng, nb, H, bs, D)).to(DEV) for _ in range(2)]
    else:
        caches = [torch.randn(nb, H, bs, D, generator=_gen(i), device=DEV).bfloat16() for i in range(2)]
    slots = torch.randint(0, nb * bs, (T,), generator=_gen(4), device=DEV)
    out = [torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    return slots, lambda: pa.pa_gather_cache(*out, slots, *caches, cache_dtype=cache_dtype), out


def _copy():
    n, H, bs, D = 1 << 18, 1, 8, 64
    caches = [torch.randn(2 * n, H, bs, D, generator=_gen(i), device=DEV).bfloat16() for i in range(2)]
    pairs = torch.stack([torch.arange(n, device=DEV), n + torch.randperm(n, generator=_gen(5), device=DEV)], 1)
    pairs = pairs.contiguous()
    return pairs, lambda: pa.pa_copy_blocks(*caches, pairs, cache_dtype="bf16"), caches


def _fp4_decode():
    """Short sequences, dealt out whole: one kernel, which signals early."""
    S, H, G, D, bs, width = 20000, 1, 8, 64, 16, 4
    rng = np.random.default_rng(6)
    caches = [torch.from_numpy(random_cache(rng, 512, H, bs, D)).to(DEV) for _ in range(2)]
    table = torch.from_numpy(rng.integers(0, 512, (S, width)).astype(np.int32)).to(DEV)
    lens = torch.from_numpy(rng.integers(1, width * bs + 1, S).astype(np.int32)).to(DEV)
    q = torch.randn(S, H * G, D, generator=_gen(7), device=DEV).bfloat16()
    out = torch.zeros_like(q)
    ws = torch.empty(pa.pa_decode_workspace_size(S, H * G, H, D, width * bs), dtype=torch.uint8, device=DEV)
    return q, lambda: pa.pa_decode(out, q, *caches, table, lens, width * bs, 0.1, cache_dtype="fp4",
                                   workspace=ws), [out]


AHEAD = {"write bf16": lambda: _write("bf16"), "write e4m3": lambda: _write("e4m3"), "write fp4": lambda: _write("fp4"),
         "gather bf16": lambda: _gather("bf16"), "gather fp4": lambda: _gather("fp4"), "copy": _copy,
         "fp4 decode": _fp4_decode}


class _Decode:
    """A decode of the older types; shared: sequences that share blocks."""

    def __init__(self, cache_dtype, shared, S=24, L=700, P=0, H=2, G=4, D=128, nb=1024):
        bs, width = 16, L // 16 + 1
        self.kw = dict(cache_dtype=cache_dtype)
        if cache_dtype == "bf16":
            self.caches = [torch.randn(nb, H, bs, D, generator=_gen(10 + i), device=DEV).bfloat16() for i in range(2)]
        else:
            self.caches = [torch.randint(-100, 100, (nb, H, bs, D), generator=_gen(10 + i), device=DEV).to(torch.int8)
                           for i in range(2)]
            self.kw.update(k_scale=0.02, v_scale=0.02)
        if shared:
            table = torch.randperm(nb, generator=_gen(12), device=DEV)[:width].expand(S, -1)
        else:
            table = torch.randint(0, nb, (S, width), generator=_gen(12), device=DEV)
        self.table, self.L = table.to(torch.int32).contiguous(), L
        self.lens = L - torch.arange(S, dtype=torch.int32, device=DEV) % 24
        self.P = P
        self.q = torch.randn(S, H * G, D, generator=_gen(13), device=DEV).bfloat16()
        self.out = torch.zeros_like(self.q)
        self.need = pa.pa_decode_workspace_size(S, H * G, H, D, L, P)

    def __call__(self, workspace):
        pa.pa_decode(self.out, self.q, *self.caches, self.table, self.lens, self.L, 0.09, partition_size=self.P,
                     workspace=workspace, **self.kw)


def _run(given, call, outputs, dec, captured, clear=True):
    kept = given.clone()
    call()
    want = [o.clone() for o in outputs]
    dec(torch.empty(dec.need, dtype=torch.uint8, device=DEV))
    want_dec = dec.out.clone()
    flat = given.view(-1).view(torch.uint8)
    assert flat.numel() >= 2 * dec.need
    at = (flat.numel() - dec.need) // 256 * 256
    ws = flat[at:at + dec.need]

    def steps():
        given.copy_(kept)
        call()
        dec(ws)

    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
    for _ in range(3):
        if clear:
            for o in outputs:
                o.zero_()
        dec.out.zero_()
        torch.cuda.synchronize()
        graph.replay() if captured else steps()
        torch.cuda.synchronize()
        for o, w in zip(outputs, want):
            assert torch.equal(o, w)
        assert torch.equal(dec.out, want_dec)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("decode", [("bf16", True), ("int8", False)])
@pytest.mark.parametrize("ahead", list(AHEAD))
def test_a_workspace_in_an_input_of_the_call_ahead(ahead, decode, captured):
    given, call, outputs = AHEAD[ahead]()
    # (a copy's sources are in its outputs)
    _run(given, call, outputs, _Decode(*decode), captured, clear=ahead != "copy")


def test_a_plan_whose_flags_are_in_the_workspace():
    """More (sequence, partition) flags than the plan keeps in shared memory."""
    given, call, outputs = _write("fp4", 131072)
    _run(given, call, outputs, _Decode("int8", False, S=66000, L=256, P=64, H=1, G=1, D=64), False)
