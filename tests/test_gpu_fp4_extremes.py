"""Four-bit attention where a few tokens take all of the weight: scores past
2^24, where only the largest (or equal ones) may count, and tokens planted in
every part of a long sequence, none of which a join may lose (GPU)."""
import numpy as np
import pytest
import torch

from oracle import fp4 as F4
from tests._fp4 import HALF_STEP, MIN_STEP, Case

pytestmark = pytest.mark.gpu


def _token(c, cache, s, h, t):
    """(codes [D / 2], scales [D / 16]) views of one token's row in the bytes."""
    tile = cache.reshape(*cache.shape[:2], -1)[c.table[s][t // c.bs], h]
    off = t % c.bs
    return (tile[:c.bs * c.D // 2].reshape(c.bs, -1)[off], tile[c.bs * c.D // 2:].reshape(-1, c.bs)[:, off])


def _copy_token(c, cache, s, h, src, dst):
    for a, b in zip(_token(c, cache, s, h, src), _token(c, cache, s, h, dst)):
        b[:] = a


def _tops(c):
    """For every query row and head: the largest score's tokens, whether the
    next score is far enough below to leave it no weight, and the values."""
    k = F4.cache_values(c.k, c.D, c.ks)
    v = F4.cache_values(c.v, c.D, c.vs)
    q = c.q.double().numpy()
    r = 0
    for s, (L, n) in enumerate(zip(c.lens, c.new)):
        pos = np.arange(L)
        blk = c.table[s][pos // c.bs]
        for j in range(n):
            m = L - n + j + 1
            for hq in range(c.H * c.G):
                h = hq // c.G
                K, V = k[blk[:m], h, pos[:m] % c.bs], v[blk[:m], h, pos[:m] % c.bs]
                sc = c.scale * (K @ q[r, hq])
                best = np.flatnonzero((K == K[sc.argmax()]).all(1))
                rest = np.delete(sc, best)
                # a score's error: D + 8 fp32 roundings of sum |q k|, and its own and its difference's
                err = abs(c.scale) * (np.abs(K) @ np.abs(q[r, hq])).max() * 2 * (c.D + 10) * 2.0 ** -23
                clear = rest.size == 0 or sc.max() - rest.max() > 2 * err + 40
                yield r, hq, clear, V[best]
            r += 1


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("q,scale", [("bf16", 2.0 ** 21), ("bf16", -2.0 ** 50), ("bf16", 2.0 ** 100), ("f16", 2.0 ** 22),
                                     ("f16", 2.0 ** 80)])
def test_one_weight_remains(op, G, D, q, scale):
    c = Case(80 + G, [700, 33, 64], G, 2, D, 16, q, scale=scale, new=None if op == "decode" else [9, 33, 1])
    for s, L in enumerate(c.lens):                             # tokens that come twice: equal weights
        for h in range(c.H):
            for t in range(0, L // 2, 3):
                _copy_token(c, c.k, s, h, t, L - 1 - t)
    g = c.device()
    getattr(c, op)(g)
    torch.cuda.synchronize()
    assert int(g.err.item()) == 0
    got = g.out.double().cpu().numpy()
    clear = total = 0
    for r, hq, ok, V in _tops(c):
        total += 1
        if not ok:
            continue
        clear += 1
        # weights of 1 or 0: a sum of at most a few rows, divided by their number, the V scale, and the output's rounding
        want, size = V.mean(0), np.abs(V).mean(0)
        off = np.abs(got[r, hq] - want)
        assert (off <= HALF_STEP[q] * np.abs(want) + MIN_STEP[q] + 2.0 ** -20 * size).all(), (r, hq, len(V))
    assert clear >= 0.9 * total


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("q,scale", [("bf16", 2.0 ** 60), ("f16", -2.0 ** 30)])
def test_equal_scores_share_the_weight(op, G, D, q, scale):
    """The largest score of every head's first query comes three times, in
    different warps, slices and pieces."""
    c = Case(85 + G, [2500, 200], G, 2, D, 16, q, scale=scale, new=None if op == "decode" else [1, 1])
    for s, L in enumerate(c.lens):
        for h in range(c.H):
            x = c.q[s, h * G].double().numpy() * np.sign(scale)
            codes = np.where(x < 0, 15, 7).astype(np.uint8)
            row, scales = _token(c, c.k, s, h, 17)
            row[:] = codes[0::2] | (codes[1::2] << 4)
            scales[:] = 0x60
            for t in (L // 2 + 1, L - 1):
                _copy_token(c, c.k, s, h, 17, t)
    g = c.device()
    getattr(c, op)(g)
    torch.cuda.synchronize()
    assert int(g.err.item()) == 0
    got = g.out.double().cpu().numpy()
    for r, hq, ok, V in _tops(c):
        if hq % G:
            continue
        assert ok and len(V) == 3
        want, size = V.mean(0), np.abs(V).mean(0)
        bound = HALF_STEP[q] * np.abs(want) + MIN_STEP[q] + 2.0 ** -20 * size
        assert (np.abs(got[r, hq] - want) <= bound).all(), (r, hq)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("lens,G,H,D,planted", [
    ([80021], 2, 1, 64, [100, 20000, 40000, 60000, 70000, 75000, 79000, 80000, 80020]),   # sixteen warps a head
    ([80021], 8, 1, 128, [7, 33000, 66000, 69000, 80001]),
    ([20011] + [1] * 19, 1, 8, 64, [3, 9000, 15000, 18000, 20010])])                      # one warp a head
def test_no_join_loses_a_piece(lens, G, H, D, planted, P):
    c = Case(90, lens, G, H, D, 32, "bf16")
    for h in range(H):
        c.q[0, h * G:(h + 1) * G] = c.q[0, h * G].clone()
        x = c.q[0, h * G].double().numpy()
        codes = np.where(x < 0, 15, 7).astype(np.uint8)        # +-6, against the query's signs
        for t in planted:
            row, scales = _token(c, c.k, 0, h, t)
            row[:] = codes[0::2] | (codes[1::2] << 4)
            scales[:] = 0x60                                   # 32: scores far above every other token's
    clear = [ok and len(V) == len(planted) for r, _, ok, V in _tops(c) if r == 0]
    assert all(clear)
    g = c.device()
    c.decode(g, P)
    torch.cuda.synchronize()
    assert int(g.err.item()) == 0
    got = g.out.double().cpu().numpy()
    for r, hq, _, V in _tops(c):
        if r:
            continue
        # equal scores, so equal weights, each 1 to the rounding of fp16
        want = V.mean(0)
        bound = HALF_STEP["bf16"] * np.abs(want) + 2.0 ** -11 * 1.01 * np.abs(V).mean(0)
        assert (np.abs(got[r, hq] - want) <= bound).all(), hq
        # the bound is tight enough: zeros, or a join without any one of the tokens, would pass it by
        assert np.median(np.abs(want) / bound) > 20
        for i in range(len(planted)):
            assert np.median(np.abs(np.delete(V, i, 0).mean(0) - want) / bound) > 5, planted[i]
