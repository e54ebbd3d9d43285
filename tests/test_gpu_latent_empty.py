"""Prefill calls none of whose sequences has a new token, between calls that
share their workspace."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, check, eps, i32
from test_gpu_latent import SCALE, expect_prefill, make_prefill

pytestmark = pytest.mark.gpu


def test_calls_without_new_tokens_leave_the_next_call_alone():
    cache, table, L, q, up, cu = make_prefill([3000, 2500, 260], [40, 300, 260], 16, 16, "bf16", 83)
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(torch.bfloat16))
    ws = torch.empty(pa.pa_latent_prefill_workspace_size(3, 16, 6000), dtype=torch.uint8, device=DEV)
    err, none = i32([0]), torch.zeros_like(cu)
    other, out = torch.full((600, 16, 128), 5.0, dtype=q.dtype, device=DEV), torch.empty(600, 16, 128, dtype=q.dtype, device=DEV)
    for _ in range(20):
        # all of these sequences are expanded, for no row
        pa.pa_latent_prefill(other, q, none, up, cache, table, L, 300, 6000, SCALE, workspace=ws, device_error=err)
        pa.pa_latent_prefill(out, q, cu, up, cache, table, L.clone(), 300, 6000, SCALE, workspace=ws, device_error=err)
    assert int(err) == 0 and bool((other == 5).all())
    check(out, want, tol)
