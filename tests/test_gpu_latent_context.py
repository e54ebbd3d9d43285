"""A prompt's rows do not depend on the tokens behind them, nor on how it is
cut into chunks."""
import pytest
import torch

from _eviction import DT, check, eps, i32
from test_gpu_latent import SCALE, expect_prefill, make_prefill, run_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("short,long", [(256, 700), (512, 513), (300, 2000), (511, 512)])
def test_first_rows_of_a_longer_sequence(short, long, dt):
    cache, table, L, q, up, cu = make_prefill([long], [long], 2, 16, dt, seed=long)
    a = run_prefill(cache, table, L, q, up, cu, SCALE, long, long)
    b = run_prefill(cache, table, i32([short]), q[:short].contiguous(), up, i32([0, short]), SCALE, short, short)
    assert torch.equal(a[:short], b)
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(DT[dt]))
    check(a, want, tol)


@pytest.mark.parametrize("cuts", [[96, 700], [256, 512, 700], [480, 700], [32, 160, 700]])
def test_chunks_of_a_prompt(cuts):
    n = cuts[-1]
    cache, table, L, q, up, cu = make_prefill([n], [n], 2, 16, "f16", seed=97)
    whole = run_prefill(cache, table, L, q, up, cu, SCALE, n, n)
    at = 0
    for end in cuts:
        got = run_prefill(cache, table, i32([end]), q[at:end].contiguous(), up, i32([0, end - at]), SCALE, end - at, end)
        assert torch.equal(got, whole[at:end]), (at, end)
        at = end
