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


@pytest.mark.parametrize("G,D", [(1, 128), (8, 64)])
@pytest.mark.parametrize("S,H", [(1, 1), (4, 4), (303, 2), (304, 2), (305, 2), (609, 1)])
def test_short_pairs_around_one_a_cta(S, H, G, D):
    """Pairs dealt out whole: fewer, as many and more than four CTAs an SM on
    152 SMs, empty sequences among them, a bad length reported."""
    rng = np.random.default_rng(S)
    lens = rng.integers(0, 513, S)
    lens[0], lens[-1] = 512, rng.integers(0, 3)
    c = Case(75, lens.tolist(), G, H, D, 16, "bf16", per_head=True)
    g = c.device()
    c.decode(g, max_len=512)
    c.check(g, f"{S} x {H}")
    want = g.out.clone()
    for bad in (-1, 10 ** 6):
        g.err.zero_()
        g.lens[-1] = bad
        g.table[-1].fill_(0)
        g.out.fill_(float("nan"))
        c.decode(g, max_len=512)
        torch.cuda.synchronize()
        assert int(g.err.item()) == 3
        assert torch.equal(g.out[:-1], want[:-1])


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("G,H,D,bs", [(1, 8, 128, 16), (2, 4, 64, 8), (8, 2, 128, 32)])
def test_sequences_that_share_blocks(op, G, H, D, bs):
    """A prefix of 2048 tokens that 24 sequences share, their tails of any
    length behind it."""
    rng = np.random.default_rng(77)
    lens = (2048 + rng.integers(0, 700, 24)).tolist()
    lens[3] = 2048
    c = Case(77, lens, G, H, D, bs, "bf16", per_head=True, new=None if op == "decode" else [3] * 24)
    c.table[:, :2048 // bs] = c.table[0, :2048 // bs]
    g = c.device()
    getattr(c, op)(g)
    c.check(g)
