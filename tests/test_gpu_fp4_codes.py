"""The four-bit write, codes and scale bytes equal to the oracle's bit for bit,
the signs of zeros among them, and the read-back's handling of slots (GPU)."""
import itertools

import numpy as np
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from oracle import fp4 as F4
from tests._fp4 import DEV
from tests.test_gpu_fp4_cache import _odd_values, _stored, _t

pytestmark = pytest.mark.gpu


def _signed_zeros(rng, x):
    """Zeros of both signs, and values that round to a zero code, among x's."""
    bits = x.view(torch.int16).clone()
    pick = torch.from_numpy(rng.random(tuple(x.shape)))
    bits[pick < 0.3] = 0
    bits[pick < 0.15] = -0x8000
    x = bits.view(x.dtype).clone()
    x[pick > 0.9] *= 2.0 ** -9
    return x


@pytest.mark.parametrize("T,H,D,bs", [(1, 1, 64, 8), (40, 3, 128, 16), (33, 5, 64, 32)])
@pytest.mark.parametrize("src", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.37, "heads"])
def test_codes_bit_for_bit(T, H, D, bs, src, scale):
    rng = np.random.default_rng(T + D)
    nb = -(-T // bs)
    sk = rng.uniform(0.01, 3, H).astype(np.float32) if scale == "heads" else np.full(H, scale, np.float32)
    arg = _t(sk) if scale == "heads" else scale
    rows = [_signed_zeros(rng, _odd_values(rng, T, H, D, src)) for _ in range(2)]
    caches = [torch.zeros(pa.fp4_cache_shape(nb, H, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pa.pa_reshape_and_cache(*(r.to(DEV) for r in rows), torch.arange(T, device=DEV), *caches, cache_dtype="fp4",
                            k_scale=arg, v_scale=arg)
    torch.cuda.synchronize()
    zeros = 0
    for r, cache in zip(rows, caches):
        codes, groups = _stored(r, sk, src)
        zeros += int((codes == 8).sum())
        got = cache.cpu().numpy()
        for t, h in itertools.product(range(T), range(H)):
            c, g = F4.unpack_tile(got[t // bs, h], bs, D)
            assert (g[t % bs] == groups[t, h]).all() and (c[t % bs] == codes[t, h]).all(), (t, h)
    assert zeros > 0


@pytest.mark.parametrize("cache_dtype", ["bf16", "int8", "fp4"])
@pytest.mark.parametrize("bad", [-2, -(1 << 40), -(1 << 63), 64, 1 << 40])
def test_gather_leaves_rows_of_bad_slots_and_reports_them(cache_dtype, bad):
    nb, H, bs, D = 4, 3, 16, 64
    shape = pa.fp4_cache_shape(nb, H, bs, D) if cache_dtype == "fp4" else (nb, H, bs, D)
    dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "fp4": torch.uint8}[cache_dtype]
    caches = [torch.full(shape, 0x22, dtype=torch.uint8, device=DEV).to(dtype) for _ in range(2)]
    out = [torch.full((5, H, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([3, bad, -1, bad, 63], device=DEV)
    pa.pa_gather_cache(*out, slots, *caches, cache_dtype=cache_dtype, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2
    for o in out:
        assert (o[1] == 7).all() and (o[3] == 7).all()         # as they were
        assert (o[2] == 0).all()                               # the padding row
        assert (o[0] != 7).all() and (o[0] != 0).all() and torch.equal(o[0], o[4])
