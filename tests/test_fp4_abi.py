"""Argument checks of the four-bit cache, the read-back and the compaction:
everything the host can see is refused before any launch (CPU)."""
import ctypes

import pytest
import torch

PTR, SLOTS = 4096, 8192    # aligned addresses that are never followed


def _lib():
    import paged_kv_cache_54_gb300 as pa
    return pa, pa.load_library()


def _desc(pa, **kw):
    d = dict(num_blocks=16, kv_heads=2, block_size=16, head_dim=64, dtype=pa.PA_FP4, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return pa.PaCacheDesc(*[d[k] for k in ("num_blocks", "kv_heads", "block_size", "head_dim", "dtype", "k_scale",
                                           "v_scale")], d.get("ks"), d.get("vs"))


BAD = [(dict(dtype=5), 1), (dict(dtype=15), 1), (dict(dtype=17), 1), (dict(k_scale=0.0), 1),
       (dict(v_scale=float("inf")), 1), (dict(v_scale=float("nan")), 1), (dict(k_scale=-1.0), 1), (dict(ks=4096), 1),
       (dict(ks=4098, vs=8192), 1), (dict(num_blocks=0), 1), (dict(block_size=24), 2), (dict(head_dim=96), 2)]


@pytest.mark.parametrize("change,status", BAD)
def test_descriptions_are_checked_by_every_call(change, status):
    pa, lib = _lib()
    d = ctypes.byref(_desc(pa, **change))
    assert lib.pa_reshape_and_cache(PTR, PTR, 1, SLOTS, 1, PTR, PTR, d, None, None) == status
    assert lib.pa_gather_cache(PTR, PTR, 1, SLOTS, 1, PTR, PTR, d, None, None) == status
    assert lib.pa_compact_blocks(PTR, PTR, d, SLOTS, 1, PTR, 1, 4, PTR, None, None) == status
    assert lib.pa_copy_blocks(PTR, PTR, d, SLOTS, 1, None, None) == status
    assert lib.pa_decode(PTR, PTR, 1, 2, 4, PTR, PTR, d, PTR, 4, PTR, 64, 1.0, 0, PTR, 1 << 30, None, None) == status
    assert lib.pa_prefill(PTR, PTR, 1, 4, PTR, 2, 4, 4, PTR, PTR, d, PTR, 4, PTR, 1.0, None, None) == status


def test_nothing_to_do_is_ok_without_pointers():
    pa, lib = _lib()
    d = ctypes.byref(_desc(pa))
    assert lib.pa_reshape_and_cache(None, None, 1, None, 0, None, None, d, None, None) == 0
    assert lib.pa_gather_cache(None, None, 1, None, 0, None, None, d, None, None) == 0
    assert lib.pa_compact_blocks(None, None, d, None, 0, None, 3, 4, None, None, None) == 0
    assert lib.pa_decode(None, None, 1, 0, 4, None, None, d, None, 4, None, 64, 1.0, 0, None, 0, None, None) == 0


def test_gather_refusals():
    pa, lib = _lib()
    d = ctypes.byref(_desc(pa))

    def rc(key=PTR, value=PTR, dst=1, slots=SLOTS, n=1, k=PTR, v=PTR, desc=d):
        return lib.pa_gather_cache(key, value, dst, slots, n, k, v, desc, None, None)

    assert rc(n=-1) == 1 and rc(key=None) == 1 and rc(value=None) == 1 and rc(slots=None) == 1
    assert rc(k=None) == 1 and rc(v=None) == 1
    assert rc(key=PTR + 8) == 1 and rc(slots=SLOTS + 4) == 1 and rc(k=PTR + 4) == 1
    assert rc(dst=pa.PA_FP4) == 2 and rc(dst=pa.PA_INT8) == 2 and rc(dst=9) == 2
    f16 = ctypes.byref(_desc(pa, dtype=pa.PA_F16))
    assert rc(desc=f16, dst=pa.PA_BF16) == 2       # a 16-bit cache is read as it is


def test_compact_refusals():
    pa, lib = _lib()
    d = ctypes.byref(_desc(pa))

    def rc(k=PTR, v=PTR, pairs=SLOTS, n=1, tables=PTR, S=1, width=4, lens=PTR):
        return lib.pa_compact_blocks(k, v, d, pairs, n, tables, S, width, lens, None, None)

    assert rc(n=-1) == 1 and rc(S=-1) == 1 and rc(width=0) == 1
    assert rc(k=None) == 1 and rc(v=None) == 1 and rc(pairs=None) == 1 and rc(tables=None) == 1 and rc(lens=None) == 1
    assert rc(k=PTR + 8) == 1 and rc(pairs=SLOTS + 4) == 1 and rc(tables=PTR + 2) == 1 and rc(lens=PTR + 1) == 1


def test_decode_and_prefill_refusals():
    pa, lib = _lib()
    d = ctypes.byref(_desc(pa))

    def dec(q=PTR, dt=1, S=2, Hq=4, P=0, ws=PTR, size=1 << 30, scale=1.0):
        return lib.pa_decode(PTR, q, dt, S, Hq, PTR, PTR, d, PTR, 4, PTR, 64, scale, P, ws, size, None, None)

    assert dec(q=PTR + 2) == 1 and dec(ws=PTR + 16) == 1 and dec(size=64) == 1 and dec(S=-1) == 1
    assert dec(Hq=3) == 1 and dec(Hq=6) == 2 and dec(Hq=32) == 2
    assert dec(dt=pa.PA_FP4) == 2 and dec(dt=pa.PA_INT8) == 2
    assert dec(P=96) == 1 and dec(P=2048) == 1 and dec(scale=float("nan")) == 1
    assert lib.pa_prefill(PTR, PTR, pa.PA_FP4, 4, PTR, 2, 4, 4, PTR, PTR, d, PTR, 4, PTR, 1.0, None, None) == 2


def test_binding_shapes():
    pa, _ = _lib()
    assert pa.fp4_cache_shape(4, 2, 16, 128) == (4, 2, 16, 72)
    kc = torch.zeros(pa.fp4_cache_shape(4, 2, 16, 128), dtype=torch.uint8)
    d = pa.cache_desc(kc, "fp4", 0.5, 0.25)
    assert (d.dtype, d.num_blocks, d.kv_heads, d.block_size, d.head_dim) == (16, 4, 2, 16, 128)
    assert (d.k_scale, d.v_scale) == (0.5, 0.25)
    with pytest.raises(ValueError):
        pa.cache_desc(torch.zeros((4, 2, 16, 64), dtype=torch.uint8), "fp4")       # not rows of nine sixteenths
    with pytest.raises(ValueError):
        pa.cache_desc(torch.zeros((4, 2, 16, 72), dtype=torch.float16), "fp4")
    with pytest.raises(ValueError):                                                # CPU tensors
        pa.pa_gather_cache(kc, kc, torch.zeros(1, dtype=torch.int64), kc, kc, cache_dtype="fp4")
    with pytest.raises(ValueError):
        pa.pa_compact_blocks(kc, kc, torch.zeros((1, 2), dtype=torch.int64), torch.zeros((1, 1), dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32), cache_dtype="fp4")
