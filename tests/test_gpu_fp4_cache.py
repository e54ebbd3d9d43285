"""The four-bit cache's write, read-back, copies, swaps and compaction on the
GPU, bit for bit against the oracle."""
import itertools

import numpy as np
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from oracle import fp4 as F4
from oracle import fp8 as F8
from oracle.cache import bits_to_f64
from tests._fp4 import DEV, DT, random_cache

pytestmark = pytest.mark.gpu


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _odd_values(rng, T, H, D, src):
    """Rows that meet every branch: ties, zeros of both signs, tiny and huge
    values, infinities and NaN."""
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    kind = rng.integers(0, 9, (T, H, D // 16))
    ties = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -0.0], np.float32)
    for t, h, g in itertools.product(range(T), range(H), range(D // 16)):
        part = x[t, h, g * 16:(g + 1) * 16]
        k = kind[t, h, g]
        if k == 0:
            part[:] = rng.permutation(ties) * rng.choice([-1, 1], 16) * 2.0 ** rng.integers(-6, 7)
        elif k == 1:
            part[:] = 0
        elif k == 2:
            part *= 2.0 ** -12
        elif k == 3:
            part *= 1e4
        elif k == 4:
            part[rng.integers(16)] = np.nan
        elif k == 5:
            part[rng.integers(16)] = np.inf
            part[rng.integers(16)] = -np.inf
        elif k == 6:
            part[:] = np.nan
        elif k == 7:
            part *= 2.0 ** rng.integers(-13, -7)
    return torch.from_numpy(x).to(DT[src])


def _stored(rows, scale, src):
    """Oracle codes [T, H, D] and scale bytes [T, H, D / 16]."""
    v = bits_to_f64(rows.view(torch.int16).numpy().view(np.uint16), src)
    T, H, D = v.shape
    codes, groups = np.zeros((T, H, D), np.uint8), np.zeros((T, H, D // 16), np.uint8)
    for t, h in itertools.product(range(T), range(H)):
        codes[t, h], groups[t, h] = F4.quantize_row(v[t, h], scale[h])
    return codes, groups


def _same_codes(a, b):
    """Codes equal, the two zeros (0 and 8) taken as one."""
    return (np.where(a == 8, 0, a) == np.where(b == 8, 0, b)).all()


CASES = [(1, 1, 64, 8, "f16", False), (3, 2, 128, 16, "bf16", False), (37, 5, 64, 32, "bf16", True),
         (64, 8, 128, 8, "f16", True), (33, 3, 128, 32, "bf16", True), (50, 40, 64, 16, "f16", False)]


@pytest.mark.parametrize("T,H,D,bs,src,per_head", CASES)
def test_write_and_read_back(T, H, D, bs, src, per_head):
    rng = np.random.default_rng(T * H + D)
    nb = -(-T // bs) + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    key, value = _odd_values(rng, T, H, D, src), _odd_values(rng, T, H, D, src)
    sk = rng.uniform(0.01, 3, H).astype(np.float32) if per_head else np.full(H, 1.0, np.float32)
    sv = rng.uniform(0.01, 3, H).astype(np.float32) if per_head else np.full(H, 0.37, np.float32)
    before = [rng.integers(0, 256, pa.fp4_cache_shape(nb, H, bs, D), dtype=np.uint8) for _ in range(2)]
    kc, vc = _t(before[0]), _t(before[1])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(cache_dtype="fp4", k_scale=_t(sk) if per_head else 1.0, v_scale=_t(sv) if per_head else float(sv[0]),
              device_error=err)
    pa.pa_reshape_and_cache(key.to(DEV), value.to(DEV), _t(slots), kc, vc, **kw)
    ko, vo = (torch.full((T, H, D), 9.0, dtype=DT[src], device=DEV) for _ in range(2))
    pa.pa_gather_cache(ko, vo, _t(slots), kc, vc, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for rows, scale, cache, was, out in ((key, sk, kc, before[0], ko), (value, sv, vc, before[1], vo)):
        codes, groups = _stored(rows, scale, src)
        got = cache.cpu().numpy()
        written = {}
        for t, slot in enumerate(slots):
            if slot >= 0:
                written.setdefault(int(slot) // bs, {})[int(slot) % bs] = t
        for b, h in itertools.product(range(nb), range(H)):
            c, g = F4.unpack_tile(got[b, h], bs, D)
            c0, g0 = F4.unpack_tile(was[b, h], bs, D)
            for off in range(bs):
                t = written.get(b, {}).get(off)
                if t is None:                                  # every other slot as it was
                    assert (c[off] == c0[off]).all() and (g[off] == g0[off]).all()
                else:
                    assert (g[off] == groups[t, h]).all(), (t, h)
                    assert _same_codes(c[off], codes[t, h]), (t, h)
        # what the rows stand for: code x group scale exactly, times the head's in fp32, rounded to 16 bits
        val = (F4.VALUES[codes] * np.repeat(F4.E4M3[groups], 16, axis=-1)).astype(np.float32) * scale[None, :, None]
        want = torch.from_numpy(val).to(DT[src])
        want[torch.from_numpy(slots) < 0] = 0
        assert torch.equal(out.cpu() + 0.0, want + 0.0)


def test_write_skips_bad_slots_and_reports_them():
    kc = torch.zeros(pa.fp4_cache_shape(2, 2, 16, 64), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([32, 1 << 40, 5], dtype=torch.int64, device=DEV)
    pa.pa_reshape_and_cache(x, x, slots, kc, vc, cache_dtype="fp4", device_error=err)
    assert int(err.item()) == 2
    v = F4.cache_values(kc.cpu().numpy(), 64)
    assert (v[0, :, 5] != 0).all() and np.count_nonzero(v) == 2 * 64
    err.zero_()
    out = torch.full_like(x, 7.0)
    pa.pa_gather_cache(out, out.clone(), slots, kc, vc, cache_dtype="fp4", device_error=err)
    assert int(err.item()) == 2
    assert (out[:2] == 7).all()                                # rows of bad slots as they were


@pytest.mark.parametrize("cache_dtype", ["f16", "bf16", "e4m3", "e5m2", "int8", "fp4"])
@pytest.mark.parametrize("bs,D,dst", [(8, 64, "f16"), (16, 128, "bf16"), (32, 64, "bf16")])
def test_gather_reads_every_cache_type(cache_dtype, bs, D, dst):
    if cache_dtype in ("f16", "bf16"):
        dst = cache_dtype
    rng = np.random.default_rng(7)
    nb, H, T = 5, 3, 61
    slots = rng.integers(-1, nb * bs, T).astype(np.int64)      # repeats and padding rows
    sk, sv = (rng.uniform(0.1, 2, H).astype(np.float32) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(cache_dtype=cache_dtype, device_error=err)
    if cache_dtype == "fp4":
        raw = [random_cache(rng, nb, H, bs, D, top=0x7E) for _ in range(2)]
        vals = [F4.cache_values(r, D).astype(np.float32) for r in raw]
        caches = [_t(r) for r in raw]
    elif cache_dtype in ("f16", "bf16"):
        caches = [torch.from_numpy(rng.standard_normal((nb, H, bs, D)).astype(np.float32)).to(DT[dst]).to(DEV)
                  for _ in range(2)]
        vals = [c.float().cpu().numpy() for c in caches]
    else:
        raw = [rng.integers(0, 256, (nb, H, bs, D), dtype=np.uint8) for _ in range(2)]
        if cache_dtype == "e4m3":
            raw = [np.where(r & 0x7F == 0x7F, 0, r) for r in raw]
        if cache_dtype == "e5m2":
            raw = [np.where(r & 0x7C == 0x7C, 0, r) for r in raw]
        if cache_dtype == "int8":
            vals = [r.view(np.int8).astype(np.float32) for r in raw]
        else:
            table = np.array([F8.decode_code(c, F8.FORMATS[cache_dtype]) for c in range(256)], np.float32)
            vals = [table[r] for r in raw]
        caches = [_t(r) for r in raw]
    if cache_dtype not in ("f16", "bf16"):
        kw.update(k_scale=_t(sk), v_scale=_t(sv))
    outs = [torch.full((T, H, D), 3.0, dtype=DT[dst], device=DEV) for _ in range(2)]
    pa.pa_gather_cache(*outs, _t(slots), *caches, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for out, v, s in zip(outs, vals, (sk, sv)):
        x = v[slots // bs, :, slots % bs]
        if cache_dtype not in ("f16", "bf16"):
            x = x * s[None, :, None]
        want = torch.from_numpy(x).to(DT[dst])
        want[torch.from_numpy(slots) < 0] = 0
        assert torch.equal(out.cpu() + 0.0, want + 0.0)


def test_copy_and_swap_move_whole_tiles():
    rng = np.random.default_rng(9)
    nb, H, bs, D = 12, 3, 8, 64
    k0, v0 = (rng.integers(0, 256, pa.fp4_cache_shape(nb, H, bs, D), dtype=np.uint8) for _ in range(2))
    kc, vc = _t(k0), _t(v0)
    pa.pa_copy_blocks(kc, vc, torch.tensor([[0, 5], [3, 6]], dtype=torch.int64, device=DEV), cache_dtype="fp4")
    host = [torch.zeros((4, H, bs, D * 9 // 16), dtype=torch.uint8).pin_memory() for _ in range(2)]
    pa.pa_swap_blocks(kc, vc, *host, torch.tensor([[5, 1], [11, 3]], dtype=torch.int64, device=DEV), "out",
                      cache_dtype="fp4")
    pa.pa_swap_blocks(kc, vc, *host, torch.tensor([[1, 9], [3, 10]], dtype=torch.int64, device=DEV), "in",
                      cache_dtype="fp4")
    torch.cuda.synchronize()
    for was, now in ((k0, kc), (v0, vc)):
        want = was.copy()
        for src, dst in ((0, 5), (3, 6), (0, 9), (11, 10)):
            want[dst] = was[src]
        assert (now.cpu().numpy() == want).all()


DTYPES = {"f16": (torch.float16, 1), "bf16": (torch.bfloat16, 1), "e4m3": (torch.uint8, 1), "int8": (torch.int8, 1)}


@pytest.mark.parametrize("cache_dtype", ["f16", "bf16", "e4m3", "e5m2", "int8", "fp4"])
@pytest.mark.parametrize("nb,S,bs,H,D", [(1, 1, 8, 1, 64), (17, 3, 16, 2, 64), (200, 9, 8, 5, 128), (96, 1, 32, 8, 128)])
def test_compact_moves_and_renames(cache_dtype, nb, S, bs, H, D):
    rng = np.random.default_rng(nb + S)
    size = 2 if cache_dtype in ("f16", "bf16") else 1
    width_bytes = D * 9 // 16 if cache_dtype == "fp4" else D * size
    raw = [rng.integers(0, 256, (nb, H, bs, width_bytes), dtype=np.uint8) for _ in range(2)]
    live = rng.permutation(nb)[: max(1, nb // 2)]
    width = len(live) + 2
    table = np.full((S, width), 3, np.int32)                   # entries behind the last block: any numbers
    table[:, 1::2] = -9
    lens = np.zeros(S, np.int32)
    for s in range(S):                                         # rows of shared and own blocks, one row empty
        n = 0 if S > 1 and s == 1 else int(rng.integers(1, len(live) + 1))
        table[s, :n] = rng.choice(live, n, replace=False)
        lens[s] = 0 if n == 0 else (n - 1) * bs + rng.integers(1, bs + 1)
    is_live = np.isin(np.arange(nb), live)
    n = len(live)
    src, dst = n + np.flatnonzero(is_live[n:]), np.flatnonzero(~is_live[:n])
    pairs = np.stack([src, dst], 1).astype(np.int64)
    code = {"f16": torch.float16, "bf16": torch.bfloat16}.get(cache_dtype)
    caches = [_t(r) if code is None else _t(r).view(code) for r in raw]
    t, err = _t(table), torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(2):                                         # the second call finds nothing left to rename
        pa.pa_compact_blocks(*caches, _t(pairs), t, _t(lens), cache_dtype=cache_dtype, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for was, now in zip(raw, caches):
        want = was.copy()
        want[dst] = was[src]
        assert (now.view(torch.uint8).cpu().numpy() == want).all()
    name = dict(zip(src.tolist(), dst.tolist()))
    want = [[name.get(int(b), int(b)) if j * bs < L else int(b) for j, b in enumerate(row)]
            for row, L in zip(table, lens)]
    assert t.cpu().numpy().tolist() == want


def test_compact_reports_and_skips_what_is_out_of_range():
    nb, H, bs, D = 10, 2, 16, 64
    rng = np.random.default_rng(3)
    raw = rng.integers(0, 256, pa.fp4_cache_shape(nb, H, bs, D), dtype=np.uint8)

    def go(pairs, table, lens):
        k, v, t = _t(raw), _t(raw), _t(np.array(table, np.int32))
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pa.pa_compact_blocks(k, v, _t(np.array(pairs, np.int64)), t, _t(np.array(lens, np.int32)), cache_dtype="fp4",
                             device_error=err)
        torch.cuda.synchronize()
        return int(err.item()), k.cpu().numpy(), t.cpu().numpy().tolist()

    e, k, t = go([[8, 99], [9, 1]], [[8, 9, 2]], [48])         # block 8 has nowhere to go and keeps its name
    assert e == 5 and t == [[8, 1, 2]] and (k[1] == raw[9]).all() and (k[8] == raw[8]).all()
    e, k, t = go([[7, 0], [1 << 35, 1]], [[7, -1, 2]], [48])   # a table entry outside the pool stays
    assert e == 5 and t == [[0, -1, 2]]
    e, k, t = go([[9, 0], [8, 1]], [[2]], [1])                 # not ascending
    assert e == 5
    e, k, t = go([[9, 0]], [[9, 9], [9, 9], [9, 9]], [33, -1, 17])
    assert e == 3 and t == [[9, 9], [9, 9], [0, 0]]
