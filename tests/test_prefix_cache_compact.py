"""Forking and compaction in the host prefix cache: the native calls against
the oracle on the same operation sequences, and the oracle's own rules (CPU)."""
import ctypes
import random

import numpy as np
import pytest

from oracle import prefix_cache as O


def _pa():
    import paged_kv_cache_54_gb300 as pa
    return pa


def _same_state(a, b, live, nb):
    assert a.stats() == b.stats()
    assert a.free_order() == b.free_order()
    for s in live:
        assert a.table(s) == b.table(s), s
    for blk in range(nb):
        assert a.ref_count(blk) == b.ref[blk]
    ok, why = b.check_invariants()
    assert ok, why


@pytest.mark.parametrize("seed", range(10))
def test_random_operations_match_the_oracle(seed):
    pa = _pa()
    rng = random.Random(500 + seed)
    bs, nb = rng.choice([1, 2, 4, 16]), rng.randrange(8, 160)
    order = rng.sample(range(nb), nb)
    nat, orc = pa.PrefixCache(nb, bs, order), O.PrefixCache(nb, bs, order)
    prefixes = [[rng.randrange(3) for _ in range(rng.randrange(0, 6 * bs))] for _ in range(3)]
    live, next_id, compactions, forks = [], 0, 0, 0

    def both(name, *args):
        res = []
        for c in (nat, orc):
            try:
                res.append(getattr(c, name)(*args))
            except (O.OutOfBlocks, pa.OutOfBlocks):
                res.append("oob")
        return res

    for step in range(300):
        op = rng.random()
        if op < 0.25 or not live:
            toks = rng.choice(prefixes) + [rng.randrange(3) for _ in range(rng.randrange(0, 3 * bs))]
            a, b = both("add_sequence", next_id, toks)
            assert a == b
            if a != "oob":
                live.append(next_id)
            next_id += 1
        elif op < 0.55:
            a, b = both("append_token", rng.choice(live), rng.randrange(3))
            assert a == b
        elif op < 0.75:
            a, b = both("fork_sequence", rng.choice(live), next_id)
            assert a == b
            if a != "oob":
                live.append(next_id)
                forks += 1
            next_id += 1
        elif op < 0.92:
            s = live.pop(rng.randrange(len(live)))
            both("free_sequence", s)
        else:
            a, b = both("compact")
            assert a.tolist() == [list(x) for x in b]
            compactions += 1
        _same_state(nat, orc, live, nb)
    assert compactions and forks


def test_compaction_leaves_kept_blocks_at_the_front():
    pa = _pa()
    c = pa.PrefixCache(32, 4, list(range(31, -1, -1)))       # blocks come from the top
    c.add_sequence(0, range(10))                             # 31, 30, 29 (the last one partial)
    c.add_sequence(1, range(100, 108))                       # 28, 27
    c.free_sequence(1)                                       # kept: both are keyed
    before = c.table(0)
    moves = c.compact()
    name = dict(moves.tolist())
    assert sorted(name) == [27, 28, 29, 30, 31] and sorted(name.values()) == [0, 1, 2, 3, 4]
    assert (np.diff(moves[:, 0]) > 0).all() and not set(name) & set(name.values())
    assert c.table(0) == [name[b] for b in before]
    assert c.free_order() == list(range(5, 32)) + [name[b] for b in (27, 28)]  # keyed ones still last
    assert c.add_sequence(2, range(100, 108)) == 8           # and still found
    assert len(c.compact()) == 0                             # nothing left to move


def test_forked_sequences_write_apart():
    pa = _pa()
    c = pa.PrefixCache(16, 4)
    c.add_sequence(0, range(6))                              # one full block, one partial
    src, dst = c.fork_sequence(0, 1)
    assert c.table(0) == [0, src] and c.table(1) == [0, dst] and c.ref_count(0) == 2
    assert c.append_token(0, 7) == src * 4 + 2 and c.append_token(1, 8) == dst * 4 + 2
    c.add_sequence(2, range(50, 58))
    assert c.fork_sequence(2, 3) is None and c.table(3) == c.table(2)
    with pytest.raises(pa.PaError):
        c.fork_sequence(0, 1)                                # child exists
    with pytest.raises(pa.PaError):
        c.fork_sequence(9, 10)                               # no such parent


def test_refusals_change_nothing():
    pa = _pa()
    lib = pa.load_library()
    c = pa.PrefixCache(4, 4, [3, 2, 1, 0])
    c.add_sequence(0, range(14))                             # all four blocks
    with pytest.raises(pa.OutOfBlocks):
        c.fork_sequence(0, 1)
    assert c.table(0) == [3, 2, 1, 0] and c.stats()["used_blocks"] == 4
    d = pa.PrefixCache(8, 4, list(range(7, -1, -1)))
    d.add_sequence(0, range(9))
    pairs = (ctypes.c_int64 * 4)(*[-7] * 4)
    assert lib.pa_prefix_cache_compact(d._h, pairs, 2) == 3  # three moves, room for two
    assert list(pairs) == [-7] * 4 and d.table(0) == [7, 6, 5]
    assert lib.pa_prefix_cache_compact(None, pairs, 2) == -1
    assert lib.pa_prefix_cache_fork_sequence(d._h, 0, 1, None) == 1
    assert lib.pa_prefix_cache_fork_sequence(None, 0, 1, pairs) == 1
