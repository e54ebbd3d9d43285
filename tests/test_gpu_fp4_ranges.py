"""Four-bit attention at the ends of what scales and queries may be, on the
GPU, against the plain attention in 64 bits."""
import numpy as np
import pytest
import torch

from tests._fp4 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("q,scale", [("bf16", 1e-20), ("bf16", -1e-20), ("bf16", 1e-36), ("bf16", 1e20),
                                     ("f16", 1e-20), ("f16", 1e-40)])
@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (4, 128), (8, 64)])
def test_tiny_queries_beside_ordinary_ones(op, q, scale, G, D):
    """Rows of 1e-30 among rows of 1: the multiplier of a row's scores neither
    underflows nor splits a warp."""
    c = Case(70, [333, 70, 5], G, 2, D, 16, q, scale=scale, new=None if op == "decode" else [200, 70, 3])
    if q == "bf16":
        c.q[::2, ::2] *= 1e-30
        c.q[1::3, 1] *= 1e-36
    if scale == 1e20:
        c.q *= 1e-20
    g = c.device()
    getattr(c, op)(g)
    c.check(g, f"{q} {scale}")
