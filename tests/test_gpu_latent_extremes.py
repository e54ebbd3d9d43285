"""Scores at the lower end of a float's range in a latent decode."""
import pytest
import torch

from _eviction import DEV, LATENT, ROW, eps, gen, i32, randn
from test_gpu_latent import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("factor", [0.86, 0.9, 0.95, 0.98])
def test_a_lone_token_takes_all_weight_however_low_its_score(factor, heads):
    """One token's softmax is one.  Scores of factor 2^128 in base 2, down from -2.9e38."""
    cache = randn(gen(heads), 1, 16, ROW).bfloat16()
    cache[0, 0, LATENT:] = 0
    cache[0, 0, LATENT] = -(2.0 ** 64)
    q = torch.zeros(1, 1, heads, ROW, dtype=torch.bfloat16, device=DEV)
    q[..., LATENT] = 2.0 ** 63
    got = run(cache, i32([[0]]), i32([1]), q, factor * 2 / 1.4426950408889634)
    want = cache[0, 0, :LATENT].double().expand(1, 1, heads, LATENT)
    assert bool(((got.double() - want).abs() <= 1.01 * eps(torch.bfloat16) * want.abs()).all())
