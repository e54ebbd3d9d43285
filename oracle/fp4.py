"""Four-bit KV codes with group scales, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A row of head_dim values is cut into groups of 16 consecutive dimensions.  A
group holds one scale g in E4M3 and 16 codes in E2M1 (sign, two exponent
bits of bias 1, one mantissa bit; no infinities, no NaN: the magnitudes 0,
0.5, 1, 1.5, 2, 3, 4, 6).  Code c stands for c * g * (the KV head's scale).

Storing x with head scale s: y = x / s in IEEE float32 (as for the one-byte
codes); g = the E4M3 value nearest to max |y| / 6 over the group (NaN left
out; ties to even; at most 448); each code is the E2M1 value nearest to
y / g (ties to even; at most 6 in magnitude), 0 for NaN, and all codes are 0
when g is 0.

A (block, head) tile is stored as the rows' codes, dimension 2j of a row in
the low half of its byte j, and then the scales as [group, token] bytes.
"""

from __future__ import annotations

import numpy as np

from . import fp8

GROUP = 16


def code_value(code: int) -> float:
    """Value of a four-bit E2M1 code, from the format definition."""
    sign, exp, man = code >> 3, (code >> 1) & 3, code & 1
    mag = man * 0.5 if exp == 0 else (1 + man * 0.5) * 2.0 ** (exp - 1)
    return -mag if sign else mag


VALUES = np.array([code_value(c) for c in range(16)])
E4M3 = np.array([fp8.decode_code(c, fp8.E4M3) for c in range(256)], dtype=np.float64)


def encode_value(r: float) -> int:
    """Nearest E2M1 code of r: the two neighbours compared, ties to the even code."""
    if np.isnan(r):
        return 0
    sign = 8 if np.signbit(r) else 0
    m = abs(float(r))
    if m >= VALUES[7]:
        return sign | 7
    hi = int(np.searchsorted(VALUES[:8], m, side="right"))  # VALUES[hi - 1] <= m < VALUES[hi]
    lo = hi - 1
    below, above = m - VALUES[lo], VALUES[hi] - m
    pick = lo if below < above or (below == above and lo % 2 == 0) else hi
    return sign | pick


def encode_scale(a: float) -> int:
    """Nearest non-negative E4M3 code of a, ties to the even code, at most 448."""
    grid = E4M3[:0x7F]                       # codes 0x00..0x7E, ascending
    if a >= grid[-1]:
        return 0x7E
    hi = int(np.searchsorted(grid, a, side="right"))
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    return lo if below < above or (below == above and lo % 2 == 0) else hi


def quantize_row(x, scale: float):
    """(codes [d] 0..15, scale bytes [d / 16]) of one row of values."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        y = (x / np.float64(np.float32(scale))).astype(np.float32).astype(np.float64)
    codes = np.zeros(x.size, dtype=np.uint8)
    groups = np.zeros(x.size // GROUP, dtype=np.uint8)
    for j in range(groups.size):
        part = y[j * GROUP:(j + 1) * GROUP]
        real = np.abs(part[~np.isnan(part)])
        groups[j] = encode_scale(real.max() / 6.0 if real.size else 0.0)
        g = E4M3[groups[j]]
        if g > 0:
            codes[j * GROUP:(j + 1) * GROUP] = [encode_value(v / g) for v in part]
    return codes, groups


def pack_tile(codes, groups) -> np.ndarray:
    """Bytes of a tile: codes [bs, d], scale bytes [bs, d / 16]."""
    codes = np.asarray(codes, dtype=np.uint8)
    pairs = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return np.concatenate([pairs.ravel(), np.asarray(groups, dtype=np.uint8).T.ravel()])


def unpack_tile(tile, bs: int, d: int):
    """(codes [bs, d], scale bytes [bs, d / 16]) of a tile's bytes."""
    tile = np.asarray(tile, dtype=np.uint8).ravel()
    pairs = tile[:bs * d // 2].reshape(bs, d // 2)
    codes = np.empty((bs, d), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = pairs & 15, pairs >> 4
    return codes, tile[bs * d // 2:].reshape(d // GROUP, bs).T.copy()


def cache_values(cache, d: int, scale=1.0) -> np.ndarray:
    """float64 values [num_blocks, kv_heads, bs, d] of a cache's bytes
    [num_blocks, kv_heads, bs, 9 d / 16]; scale: one number or one per head."""
    cache = np.asarray(cache, dtype=np.uint8)
    nb, H, bs, _ = cache.shape
    tile = cache.reshape(nb, H, -1)
    pairs = tile[..., :bs * d // 2].reshape(nb, H, bs, d // 2)
    v = np.empty((nb, H, bs, d))
    v[..., 0::2], v[..., 1::2] = VALUES[pairs & 15], VALUES[pairs >> 4]
    g = E4M3[tile[..., bs * d // 2:].reshape(nb, H, d // GROUP, bs)].transpose(0, 1, 3, 2)
    s = np.broadcast_to(np.asarray(scale, dtype=np.float32).astype(np.float64), (H,))
    return v * np.repeat(g, GROUP, axis=-1) * s[None, :, None, None]
