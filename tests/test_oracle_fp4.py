"""The four-bit oracle is pinned to the format definitions, brute force and
hand-worked cases (CPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle import fp4 as F4


def test_code_values_are_e2m1():
    assert F4.VALUES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert (F4.VALUES[8:] == -F4.VALUES[:8]).all()


def test_every_code_is_its_own_nearest():
    for c in range(16):
        assert F4.encode_value(F4.code_value(c)) == (c if c != 8 else 8)


@pytest.mark.parametrize("value,want", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0),
                                        (3.5, 4.0), (5.0, 4.0), (7.0, 6.0), (1e30, 6.0), (np.inf, 6.0)])
def test_ties_go_to_even_and_large_values_saturate(value, want):
    for sign in (1, -1):
        assert F4.VALUES[F4.encode_value(sign * value)] == sign * want


def test_nearest_by_brute_force():
    rng = np.random.default_rng(1)
    for r in rng.uniform(-7, 7, 5000):
        got = F4.VALUES[F4.encode_value(r)]
        assert abs(got - np.clip(r, -6, 6)) == np.abs(F4.VALUES - np.clip(r, -6, 6)).min()


def test_scales_match_torch_rounding_and_saturate():
    rng = np.random.default_rng(2)
    a = np.concatenate([rng.uniform(0, 500, 4000), 2.0 ** rng.uniform(-14, 9, 4000), F4.E4M3[:0x7F],
                        (F4.E4M3[:0x7E] + F4.E4M3[1:0x7F]) / 2]).astype(np.float32)
    want = torch.from_numpy(np.minimum(a, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [F4.encode_scale(float(v)) for v in a] == want.tolist()


def test_tiles_round_trip():
    rng = np.random.default_rng(3)
    for bs, d in itertools.product((8, 16, 32), (64, 128)):
        codes = rng.integers(0, 16, (bs, d), dtype=np.uint8)
        groups = rng.integers(0, 127, (bs, d // 16), dtype=np.uint8)
        tile = F4.pack_tile(codes, groups)
        assert tile.size == bs * d * 9 // 16
        c, g = F4.unpack_tile(tile, bs, d)
        assert (c == codes).all() and (g == groups).all()
        v = F4.cache_values(tile.reshape(1, 1, bs, -1), d, 0.5)[0, 0]
        t, i = 3, 37                                    # one value by hand
        assert v[t, i] == F4.VALUES[codes[t, i]] * F4.E4M3[groups[t, i // 16]] * 0.5
        assert tile[t * d // 2 + i // 2] >> (4 * (i % 2)) & 15 == codes[t, i]
        assert tile[bs * d // 2 + (i // 16) * bs + t] == groups[t, i // 16]


def test_quantised_rows_are_near_and_planted_mistakes_are_not():
    rng = np.random.default_rng(4)
    x = rng.standard_normal(128) * 3
    codes, groups = F4.quantize_row(x, 0.125)
    v = F4.VALUES[codes] * np.repeat(F4.E4M3[groups], 16) * 0.125
    # a code is off by at most half a step (1 of 6 near the top), the top by
    # the scale's own rounding (1/16 of it) besides
    top = np.abs(x).reshape(-1, 16).max(1).repeat(16)
    assert (np.abs(v - x) <= top / 6 * (1 + 1 / 16) + 1e-12).all()
    swapped = (codes[0::2].astype(int) << 4 | codes[1::2]).astype(np.uint8)   # halves exchanged
    assert (swapped != F4.pack_tile(codes[None], groups[None])[:64]).any()


def test_odd_rows():
    zeros = F4.quantize_row(np.zeros(64), 1.0)
    assert not zeros[0].any() and not zeros[1].any()
    tiny = F4.quantize_row(np.full(64, 1e-4), 1.0)        # the scale rounds to zero
    assert not tiny[0].any() and not tiny[1].any()
    x = np.zeros(64)
    x[3], x[5], x[20] = np.nan, 6.0, np.inf
    codes, groups = F4.quantize_row(x, 1.0)
    assert codes[3] == 0 and F4.VALUES[codes[5]] == 6.0 and F4.E4M3[groups[0]] == 1.0
    assert codes[20] == 7 and F4.E4M3[groups[1]] == 448.0
