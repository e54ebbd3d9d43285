"""Many short sequences in one latent decode, around the number up to which
they are not split, and rows around the borders of the joins' variants."""
import pytest
import torch

from _eviction import DT, check, eps
from test_gpu_latent import SCALE, expect, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,new", [(152, 128, 1), (153, 128, 1), (76, 128, 2), (77, 100, 2), (304, 16, 1), (305, 16, 1),
                                            (306, 16, 4), (400, 3, 1)])
def test_many_short_sequences(seqs, heads, new):
    lens = [(s * 37) % 201 for s in range(seqs)]
    cache, table, L, q = make(lens, new, heads, 16, "bf16", seqs + heads)
    got = run(cache, table, L, q, SCALE, max_len=256)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    check(got, want, tol)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,heads", [([3000], 76), ([3000], 77), ([3000, 700], 38), ([3000, 700, 1], 26), ([900] * 8, 128),
                                        ([900] * 8 + [300], 120), ([700] * 66, 16), ([700] * 67, 16)])
def test_rows_around_the_joins_borders(lens, heads, dt):
    cache, table, L, q = make(lens, 1, heads, 32, dt, len(lens) + heads)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, 32, SCALE, eps(DT[dt]))
    check(got, want, tol)
