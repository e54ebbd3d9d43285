"""Drafted tokens that are not finite: a row of pa_latent_decode is a function
of the tokens that it sees, whatever the later ones hold."""
import math

import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, DT, LATENT, attend, eps, i32, rows_of
from test_gpu_latent import SCALE, expect, make, run

pytestmark = pytest.mark.gpu

BAD = {"inf": {7: math.inf}, "-inf": {300: -math.inf}, "nan": {511: math.nan, 0: math.nan}, "key": {530: math.inf},
       "both": {40: math.inf, 41: -math.inf, 200: math.nan}}


def put(cache, table, s, token, bs, what):
    for d, x in BAD[what].items():
        cache[int(table[s, token // bs]), token % bs, d] = x


def same(got, want, tol):
    """Not-a-number and infinite where the definition is, within the tolerance elsewhere."""
    got = got.double()
    assert bool((torch.isnan(got) == torch.isnan(want)).all()), "not-a-number in other places"
    inf = torch.isinf(want)
    assert bool((got[inf] == want[inf]).all())
    ok = torch.isfinite(want)
    assert bool(((got - want).abs() <= tol)[ok].all()), float((got - want).abs()[ok].max())


def definition(cache, table, L, q, bs, e):
    """As `expect`; the tolerance is that of the tokens that are finite (one that is not leaves a row its other
    tokens' sums, where its weight is zero, or nothing finite)."""
    S, n, H, _ = q.shape
    o = torch.zeros(S, n, H, LATENT, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    for s, length in enumerate(L.tolist()):
        x = rows_of(cache, table[s], length, bs)
        for j in range(n):
            see = length - (n - 1 - j)
            if see > 0:
                o[s, j] = attend(q[s, j].double(), x[:see], x[:see, :LATENT], SCALE, e)[0]
                y = x[:see][torch.isfinite(x[:see]).all(-1)]
                if len(y):
                    tol[s, j] = attend(q[s, j].double(), y, y[:, :LATENT], SCALE, e)[1]
    return o, tol


# lens, new tokens, heads, block, bound on the lengths (None: their largest).  Lengths around the tiles of 64 and 128
# tokens, so that the drafted tokens lie on both sides of a tile's end; rows for each of the kernels; whole and split.
SHAPES = [
    ([100, 64, 128, 66, 130], 2, 8, 16, None),
    ([66, 5, 130, 64], 5, 3, 8, None),
    ([127, 128, 129, 65], 2, 16, 32, None),
    ([66, 5, 130, 64], 4, 8, 16, 5000),
    ([9000, 70], 3, 16, 16, None),
    ([9000, 66], 3, 20, 16, None),
    ([100, 128, 130, 256], 2, 64, 16, None),
    ([128, 131, 5, 200], 4, 128, 16, None),
    ([128, 131, 256], 40, 4, 8, 5000),
    ([9000, 130], 5, 40, 32, None),
    ([4000, 4224], 3, 128, 16, None),
]


@pytest.mark.parametrize("what", list(BAD))
@pytest.mark.parametrize("lens,new,heads,bs,most", SHAPES)
def test_a_drafted_token_reaches_no_row_before_it(lens, new, heads, bs, most, what):
    for dt in ("f16", "bf16"):
        cache, table, L, q = make(lens, new, heads, bs, dt, seed=len(lens) * 31 + heads)
        for s, n in enumerate(lens):
            put(cache, table, s, n - 1, bs, what)                  # the last drafted token
            if s == 1 and new > 2:
                put(cache, table, s, n - 2, bs, "both")
        got = run(cache, table, L, q, SCALE, max_len=most)
        want, tol = definition(cache, table, L, q, bs, eps(DT[dt]))
        assert bool(torch.isfinite(want[:, :1]).all())             # the first row meets none of them
        same(got, want, tol)


@pytest.mark.parametrize("heads", [16, 128])
def test_finite_drafts_are_as_before(heads):
    cache, table, L, q = make([64, 128, 130, 3000], 4, heads, 16, "f16", 3)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.float16))
    same(got, want, tol)


@pytest.mark.parametrize("heads", [16, 128])
def test_a_bad_token_under_a_minus_infinite_score(heads):
    """The token's weight is zero; its dimension is 0 * infinity in the rows that see it, the others stay finite."""
    cache, table, L, q = make([130], 3, heads, 16, "bf16", 5)
    put(cache, table, 0, 128, 16, "inf")
    q[..., 7] = -q[..., 7].abs() - 0.1
    got = run(cache, table, L, q, SCALE)
    assert bool(torch.isfinite(got[:, 0]).all())
    assert bool(torch.isnan(got[:, 1:, :, 7]).all())
    keep = [d for d in range(LATENT) if d != 7]
    assert bool(torch.isfinite(got[:, 1:, :, keep]).all())
    want, tol = definition(cache, table, L, q, 16, eps(torch.bfloat16))
    same(got, want, tol)


def test_replayed_with_a_bad_draft():
    cache, table, L, q = make([130, 66], 4, 16, 16, "bf16", 9)
    ws = torch.empty(pa.pa_latent_decode_workspace_size(2, 4, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty(2, 4, 16, LATENT, dtype=torch.bfloat16, device=DEV)
    pa.pa_latent_decode(out, q, cache, table, L, 1000, SCALE, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_latent_decode(out, q, cache, table, L, 1000, SCALE, workspace=ws)
    put(cache, table, 0, 129, 16, "nan")
    L.copy_(i32([130, 60]))
    graph.replay()
    want, tol = definition(cache, table, L, q, 16, eps(torch.bfloat16))
    same(out, want, tol)
