"""Rows of a latent write that lie further apart than 32-bit indexes reach."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, LATENT, ROW, gen, i32, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [(1 << 31) + 8, 1 << 20])
def test_rows_far_apart(stride):
    tokens = 3
    far = torch.empty((tokens - 1) * stride + ROW, dtype=torch.bfloat16, device=DEV)
    rows = far.as_strided((tokens, ROW), (stride, 1))
    rows.copy_(randn(gen(1), tokens, ROW).bfloat16())
    cache, err = torch.zeros(4, 16, ROW, dtype=torch.bfloat16, device=DEV), i32([0])
    slots = torch.tensor([63, 0, 17], device=DEV)
    pa.pa_latent_write(rows[:, :LATENT], rows[:, LATENT:], slots, cache, device_error=err)
    want = torch.zeros_like(cache)
    want.view(-1, ROW)[slots] = rows
    assert int(err) == 0 and torch.equal(cache, want)
