"""The latent cache on the GPU: rows written through a slot mapping, and
absorbed attention of one or a few new tokens, against the definition in 64
bits."""
import math

import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, DT, LATENT, ROPE, ROW, attend, check, eps, gen, i32, randn, rows_of, tables

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("tokens", [1, 3, 64, 1021])
@pytest.mark.parametrize("dt,bs", [("f16", 8), ("bf16", 16), ("bf16", 32)])
def test_write_is_a_copy(tokens, dt, bs):
    g = gen(tokens + bs)
    nb = -(-tokens // bs) + 2
    both = randn(g, tokens, ROW + 64).to(DT[dt])      # rows of a wider projection
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:tokens]
    slots[::5] = -1
    cache = randn(g, nb, bs, ROW).to(DT[dt])
    want = cache.clone()
    keep = slots >= 0
    want.view(-1, ROW)[slots[keep]] = both[keep, :ROW]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_latent_write(both[:, :LATENT], both[:, LATENT:ROW], slots, cache, device_error=err)
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16)) and int(err) == 0
    cache2 = torch.zeros_like(cache)
    pa.pa_latent_write(both[:, :LATENT].contiguous(), both[:, LATENT:ROW].contiguous(), slots, cache2)
    assert torch.equal(cache2.view(-1, ROW)[slots[keep]].view(torch.int16), both[keep, :ROW].view(torch.int16))


def test_write_reports_slots_outside_the_cache():
    cache = torch.zeros(2, 16, ROW, dtype=torch.float16, device=DEV)
    x = torch.ones(4, ROW, dtype=torch.float16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([32, -2, 5, 2 ** 40], device=DEV)
    pa.pa_latent_write(x[:, :LATENT], x[:, LATENT:], slots, cache, device_error=err)
    assert int(err) == 2
    assert float(cache.float().sum()) == ROW and float(cache.view(-1, ROW)[5].float().sum()) == ROW


def test_write_without_tokens_and_past_four_gigabytes():
    nb = (1 << 32) // (32 * ROW * 2) + 40
    cache = torch.zeros(nb, 32, ROW, dtype=torch.bfloat16, device=DEV)
    x = randn(gen(1), 3, ROW).bfloat16()
    pa.pa_latent_write(x[:0, :LATENT], x[:0, LATENT:], torch.zeros(0, dtype=torch.int64, device=DEV), cache)
    slots = torch.tensor([nb * 32 - 1, 0, nb * 32 - 40], device=DEV)
    pa.pa_latent_write(x[:, :LATENT], x[:, LATENT:], slots, cache)
    assert torch.equal(cache.view(-1, ROW)[slots], x)


# ---------------------------------------------------------------- decode
def make(lens, new, heads, bs, dt, seed, width=None):
    g = gen(seed)
    table, nb, _ = tables(lens, bs, seed, width=width)
    cache = torch.full((nb, bs, ROW), float("nan"), dtype=DT[dt], device=DEV)
    for s, n in enumerate(lens):   # rows behind a sequence's end stay NaN
        for b in range(-(-n // bs)):
            m = min(bs, n - b * bs)
            cache[int(table[s, b]), :m] = randn(g, m, ROW).to(DT[dt])
    q = torch.cat((0.4 * randn(g, len(lens), new, heads, LATENT), randn(g, len(lens), new, heads, ROPE)), -1)
    return cache, table, i32(lens), q.to(DT[dt])


def expect(cache, table, lens, q, bs, scale, e):
    S, n, H, _ = q.shape
    o = torch.zeros(S, n, H, LATENT, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    for s, L in enumerate(lens.tolist()):
        x = rows_of(cache, table[s], L, bs)
        for j in range(n):
            see = L - (n - 1 - j)
            if see > 0:
                o[s, j], tol[s, j], _, _ = attend(q[s, j].double(), x[:see], x[:see, :LATENT], scale, e)
    return o, tol


def run(cache, table, lens, q, scale, max_len=None, **kw):
    out = torch.full(q.shape[:-1] + (LATENT,), float("nan"), dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_latent_decode(out, q, cache, table, lens, int(lens.max()) if max_len is None else max_len, scale,
                        device_error=err, **kw)
    assert int(err) == 0
    return out


SCALE = 1.0 / math.sqrt(192)
SHAPES = [
    # lens, new tokens, heads, block
    ([1], 1, 16, 16),
    ([64], 1, 16, 16),
    ([65, 63, 128], 1, 16, 8),
    ([1, 2, 7, 0, 33, 100], 1, 5, 16),
    ([300, 1, 129], 1, 1, 32),
    ([77, 500], 1, 20, 8),
    ([77, 500, 64], 1, 64, 16),
    ([130, 1, 700], 1, 128, 32),
    ([1000, 3], 2, 16, 16),
    ([2, 1, 0, 200], 4, 16, 32),       # rows that see nothing
    ([90, 257], 3, 20, 16),
    ([400], 5, 128, 8),
    ([0, 0], 1, 16, 16),
    ([5000], 1, 16, 16),
    ([3000, 4000, 200], 1, 64, 32),
    ([128, 256], 1, 128, 16),
    ([129, 0, 2000, 64], 1, 100, 8),   # 128 rows a tile, some of them none
    ([3000, 1], 2, 96, 32),
    ([9000, 300], 1, 128, 16),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new,heads,bs", SHAPES)
def test_decode_matches_the_definition(lens, new, heads, bs, dt):
    cache, table, L, q = make(lens, new, heads, bs, dt, seed=len(lens) * 100 + heads)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, bs, SCALE, eps(DT[dt]))
    check(got, want, tol)


def test_decode_of_many_sequences_of_many_lengths():
    lens = [(37 * s * s) % 700 for s in range(300)]
    cache, table, L, q = make(lens, 1, 16, 16, "bf16", 7)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    check(got, want, tol)


@pytest.mark.parametrize("heads", [32, 128])
@pytest.mark.parametrize("factor", [0.0, -3.0, 40.0])
def test_decode_scales(factor, heads):
    # (40 times the usual scale: maxima rise by far more than 2^8 on the way, and few tokens take all of the weight)
    cache, table, L, q = make([700, 64, 3], 1, heads, 16, "f16", 11)
    got = run(cache, table, L, q, SCALE * factor)
    want, tol = expect(cache, table, L, q, 16, SCALE * factor, eps(torch.float16))
    check(got, want, tol)


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_with_rising_scores(heads):
    """Every tile's scores lie far above the last one's."""
    cache, table, L, q = make([900], 1, heads, 16, "bf16", 13)
    n = torch.arange(900, device=DEV)
    rows = cache[table[0].long()].view(-1, ROW)
    rows[:900] = (rows[:900].float() * (n[:, None] / 100.0)).bfloat16()
    cache[table[0].long()] = rows.view(-1, 16, ROW)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    check(got, want, tol)


def test_decode_infinities_stay_in_their_rows():
    cache, table, L, q = make([100, 100], 1, 16, 16, "f16", 17)
    q[0, 0, 3, 0] = float("nan")
    cache[int(table[1, 2]), 5, 7] = float("inf")
    out = run(cache, table, L, q, SCALE)
    assert torch.isnan(out[0, 0, 3]).all()
    clean = [h for h in range(16) if h != 3]
    want, tol = expect(cache, table[:1], L[:1], q[:1], 16, SCALE, eps(torch.float16))
    check(out[0, 0, clean], want[0, 0, clean], tol[0, 0, clean])
    assert not torch.isfinite(out[1]).all(-1).any()   # every row of the sequence meets the infinity


def test_decode_three_dimensional_queries_wider_tables_and_bounds():
    cache, table, L, q = make([200, 70], 1, 16, 16, "bf16", 19, width=40)
    a = run(cache, table, L, q, SCALE)
    out = torch.empty(2, 16, LATENT, dtype=torch.bfloat16, device=DEV)
    pa.pa_latent_decode(out, q[:, 0].contiguous(), cache, table, L, 640, SCALE)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    check(a, want, tol)
    check(out, want[:, 0], tol[:, 0])


def offset(t, elements=8):
    """The tensor's values in a tensor that lies 16 bytes further on."""
    x = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)[elements:].view(t.shape)
    return x.copy_(t)


@pytest.mark.parametrize("heads", [16, 128])
def test_tensors_aligned_to_16_bytes_only(heads):
    cache, table, L, q = make([300, 70], 1, heads, 16, "bf16", 21)
    cache, q, out = offset(cache), offset(q), offset(torch.empty(2, 1, heads, LATENT, dtype=q.dtype, device=DEV))
    assert out.data_ptr() % 32 == 16
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    for most in (300, 5000):
        out.fill_(float("nan"))
        pa.pa_latent_decode(out, q, cache, table, L, most, SCALE)
        check(out, want, tol)
    new = torch.zeros_like(cache)
    slots = torch.arange(7, device=DEV)
    pa.pa_latent_write(cache.view(-1, ROW)[:7, :LATENT], cache.view(-1, ROW)[:7, LATENT:], slots, new)
    assert torch.equal(new.view(-1, ROW)[:7].view(torch.int16), cache.view(-1, ROW)[:7].view(torch.int16))


def test_prefill_tensors_aligned_to_16_bytes_only():
    cache, table, L, q, up, cu = make_prefill([200, 30], [140, 30], 3, 16, "f16", 22)
    cache, q, up, out = (offset(x) for x in (cache, q, up, torch.zeros(170, 3, 128, dtype=q.dtype, device=DEV)))
    pa.pa_latent_prefill(out, q, cu, up, cache, table, L, 140, 230, SCALE)
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(torch.float16))
    check(out, want, tol)


def test_decode_reports_bad_lengths_and_blocks():
    cache, table, L, q = make([100, 100, 100], 1, 16, 16, "f16", 23)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((3, 1, 16, LATENT), 7.0, dtype=torch.float16, device=DEV)
    bad = L.clone()
    bad[1] = 101
    pa.pa_latent_decode(out, q, cache, table, bad, 100, SCALE, device_error=err)
    assert int(err) == 3 and float(out[1].abs().sum()) == 0
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.float16))
    check(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
    err.zero_()
    cache[0] = 0                       # (what the bad entry is read as; it may be a sequence's own block too)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.float16))
    t = table.clone()
    t[2, 3] = 10 ** 6
    pa.pa_latent_decode(out, q, cache, t, L, 100, SCALE, device_error=err)
    assert int(err) == 1
    check(out[:2], want[:2], tol[:2])


def test_decode_past_four_gigabytes():
    bs, nb = 32, (1 << 32) // (32 * ROW * 2) + 200
    cache = torch.zeros(nb, bs, ROW, dtype=torch.bfloat16, device=DEV)
    g = gen(29)
    table = i32([[nb - 1, 0, nb - 117, 5]])
    cache[table[0].long()] = randn(g, 4, bs, ROW).bfloat16()
    q = randn(g, 1, 1, 16, ROW).bfloat16()
    L = i32([4 * bs - 3])
    got = run(cache, table, L, q, SCALE * 0.5)
    want, tol = expect(cache, table, L, q, bs, SCALE * 0.5, eps(torch.bfloat16))
    check(got, want, tol)


def test_decode_captured_and_replayed_on_another_stream():
    cache, table, L, q = make([300, 4000, 0, 77], 2, 16, 16, "bf16", 31)
    ws = torch.empty(pa.pa_latent_decode_workspace_size(4, 2, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty(4, 2, 16, LATENT, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pa.pa_latent_decode(out, q, cache, table, L, 4096, SCALE, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_latent_decode(out, q, cache, table, L, 4096, SCALE, workspace=ws)
    ws.random_()
    L.copy_(i32([299, 3001, 0, 60]))   # no longer than the blocks they have
    q.copy_(randn(gen(37), *q.shape) * 0.5)
    out.fill_(float("nan"))
    graph.replay()
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
    check(out, want, tol)


@pytest.mark.parametrize("heads", [2, 16, 80])
def test_decode_of_more_than_a_thousand_sequences(heads):
    lens = [(s * 29) % 130 if s % 5 else 0 for s in range(1100)]
    lens[3], lens[700], lens[1099] = 9000, 5000, 7000     # in many pieces
    cache, table, L, q = make(lens, 1, heads, 8, "bf16", 57)
    got = run(cache, table, L, q, SCALE)
    want, tol = expect(cache, table, L, q, 8, SCALE, eps(torch.bfloat16))
    check(got, want, tol)


@pytest.mark.parametrize("heads,new", [(16, 1), (40, 1), (72, 2)])
def test_decode_of_short_sequences_some_of_them_empty(heads, new):
    lens = [0, 40, 0, 256, 1, 0, 64]     # none is split
    cache, table, L, q = make(lens, new, heads, 16, "f16", 54)
    got = run(cache, table, L, q, SCALE, max_len=256)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.float16))
    check(got, want, tol)


@pytest.mark.parametrize("lens,new,heads", [([5000, 700], 4, 128), ([900, 2500], 77, 128), ([700, 900], 3, 16)])
def test_decode_stays_within_its_workspace(lens, new, heads):
    # several row tiles that divide the shares among them, and more row tiles than shares
    cache, table, L, q = make(lens, new, heads, 16, "bf16", 53)
    need = pa.pa_latent_decode_workspace_size(len(lens), new, heads)
    ws = torch.full((need + (1 << 20),), 0x5a, dtype=torch.uint8, device=DEV)
    got = run(cache, table, L, q, SCALE, workspace=ws[:need])
    assert bool((ws[need:] == 0x5a).all())
    for h in {0, heads // 2, heads - 1}:
        want, tol = expect(cache, table, L, q[:, :, h:h + 1], 16, SCALE, eps(torch.bfloat16))
        check(got[:, :, h:h + 1], want, tol)


# ---------------------------------------------------------------- prefill
def make_prefill(lens, new, heads, bs, dt, seed):
    cache, table, L, _ = make(lens, 1, 1, bs, dt, seed)
    g = gen(seed + 1)
    T = sum(new)
    q = randn(g, T, heads, 192).to(DT[dt])
    up = (randn(g, heads, 256, LATENT) / math.sqrt(LATENT)).to(DT[dt])
    cu = i32([sum(new[:s]) for s in range(len(new) + 1)])
    return cache, table, L, q, up, cu


def expect_prefill(cache, table, lens, q, up, cu, bs, scale, e):
    """The definition, and the bound of `attend` with what the expansion adds:
    keys and values are rounded to the cache's type (eps / 2 of each) after
    sums of 512 products in 32 bits (2^-24 a partial sum, 512 of them)."""
    o = torch.zeros(q.shape[0], q.shape[1], 128, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    cu = cu.tolist()
    for s, L in enumerate(lens.tolist()):
        x = rows_of(cache, table[s], L, bs)
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        hidden = torch.arange(L, device=DEV)[None] > (L - n + torch.arange(n, device=DEV))[:, None]
        for h in range(q.shape[1]):
            u = up[h].double()
            kv, kv_size = x[:, :LATENT] @ u.T, x[:, :LATENT].abs() @ u.abs().T
            off = e / 2 * kv.abs() + 512 * 2.0 ** -24 * kv_size
            key, qq = torch.cat((kv[:, :128], x[:, LATENT:]), 1), q[cu[s]:cu[s + 1], h].double()
            w = torch.softmax((qq @ key.T * scale).masked_fill(hidden, -math.inf), -1)
            v = kv[:, 128:]
            out, spread = w @ v, w @ v.abs()
            # scores: the keys' error, the sum of 192 products, the exponential
            d = abs(scale) * ((qq[:, :128].abs() @ off[:, :128].T) + 194 * 2.0 ** -24 * (qq.abs() @ key.abs().T))
            d = d.masked_fill(hidden, 0).amax(-1, keepdim=True) + 2.0 ** -21
            o[cu[s]:cu[s + 1], h] = out
            tol[cu[s]:cu[s + 1], h] = e / 2 * (out.abs() + spread) * 1.01 + 2 * d * spread + w @ off[:, 128:]
    return o, tol


def run_prefill(cache, table, lens, q, up, cu, scale, max_new, tokens, **kw):
    out = torch.full((q.shape[0], q.shape[1], 128), float("nan"), dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_latent_prefill(out, q, cu, up, cache, table, lens, max_new, tokens, scale, device_error=err, **kw)
    assert int(err) == 0
    return out


PREFILL = [
    # lens, new tokens, heads, block
    ([1], [1], 1, 16),
    ([128], [128], 2, 8),
    ([129, 64], [129, 1], 3, 16),
    ([100, 300, 0, 17], [3, 257, 0, 17], 4, 32),
    ([1000], [600], 2, 16),
    ([511, 512, 513], [255, 256, 257], 2, 32),
    ([2000, 5], [40, 5], 16, 8),
    ([70] * 20, [2] * 20, 5, 16),
    ([600, 40, 1000, 257, 300] * 6, [300, 1, 513, 257, 128] * 6, 7, 16),   # several items a block
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new,heads,bs", PREFILL)
def test_prefill_matches_the_definition(lens, new, heads, bs, dt):
    cache, table, L, q, up, cu = make_prefill(lens, new, heads, bs, dt, seed=sum(lens) + heads)
    got = run_prefill(cache, table, L, q, up, cu, SCALE, max(new), sum(lens))
    want, tol = expect_prefill(cache, table, L, q, up, cu, bs, SCALE, eps(DT[dt]))
    check(got, want, tol)


@pytest.mark.parametrize("seqs", [127, 128, 129, 300])
def test_prefill_and_decode_of_many_short_sequences(seqs):
    lens = [(s * 31) % 150 if s % 4 else 0 for s in range(seqs)]
    lens[-1] = 300
    new = [min(n, s % 5) for s, n in enumerate(lens)]
    cache, table, L, q, up, cu = make_prefill(lens, new, 2, 16, "f16", 59)
    got = run_prefill(cache, table, L, q, up, cu, SCALE, max(new), sum(lens))
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(torch.float16))
    check(got, want, tol)
    for heads in (3, 70):
        cache, table, L, q = make(lens, 1, heads, 16, "f16", 60)
        want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.float16))
        check(run(cache, table, L, q, SCALE), want, tol)


@pytest.mark.parametrize("factor", [0.0, -2.0, 30.0])
def test_prefill_scales(factor):
    cache, table, L, q, up, cu = make_prefill([700, 64], [300, 64], 2, 16, "f16", 51)
    got = run_prefill(cache, table, L, q, up, cu, SCALE * factor, 300, 764)
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE * factor, eps(torch.float16))
    check(got, want, tol)


def test_prefill_values_of_all_magnitudes():
    """Groups of 32 tokens whose values lie many powers of two apart, up and down, beside fp16's range."""
    L = [400, 90]
    cache, table, lens, q, up, cu = make_prefill(L, [300, 90], 2, 16, "bf16", 55)
    up[:, :128] = 0                                          # (scores from the rotary part alone)
    power = [0, 40, -30, 17, 16, -20, 60, 0, 61, 3, -60, 30, 0]
    for s, n in enumerate(L):
        for b in range(-(-n // 16)):
            cache[int(table[s, b]), :, :LATENT] *= 2.0 ** power[(b // 2 + s) % len(power)]
    cache[torch.isnan(cache)] = 0                            # (rows behind the ends; the factor of 0 * NaN)
    got = run_prefill(cache, table, lens, q, up, cu, SCALE, 300, 490)
    want, tol = expect_prefill(cache, table, lens, q, up, cu, 16, SCALE, eps(torch.bfloat16))
    # beside that: a value is a step of 2^-25 of its group's largest off (times 2^-13 of its scaling), a weight 2^-25 in
    # the units of the largest group a row follows, over all keys
    big = torch.zeros_like(want)
    for s, n in enumerate(L):
        x = rows_of(cache, table[s], n, 16)
        for h in range(2):
            v = (x[:, :LATENT] @ up[h, 128:].double().T).abs().amax(-1)
            seen = torch.cummax(torch.cat([v[i:i + 32].max().expand(len(v[i:i + 32])) for i in range(0, n, 32)]), 0).values
            m = int(cu[s + 1] - cu[s])
            big[cu[s]:cu[s + 1], h] = seen[n - m:, None] * (torch.arange(n - m, n, device=DEV)[:, None] + 64)
    check(got, want, tol + 2.0 ** -24 * big)


def test_prefill_bounds_above_and_rows_left_alone():
    """Bounds larger than the lengths, rows of q behind the last sequence, a wider table."""
    cache, table, L, q, up, cu = make_prefill([200, 30], [140, 30], 2, 16, "bf16", 53)
    q = torch.cat((q, torch.full_like(q[:9], float("nan"))))
    table = torch.cat((table, torch.full_like(table, -3)), 1).contiguous()
    out = torch.full((q.shape[0], 2, 128), 5.0, dtype=q.dtype, device=DEV)
    pa.pa_latent_prefill(out, q, cu, up, cache, table, L, 1000, 5000, SCALE)
    want, tol = expect_prefill(cache, table, L, q[:170], up, cu, 16, SCALE, eps(torch.bfloat16))
    check(out[:170], want, tol)
    assert bool((out[170:] == 5.0).all())


def test_prefill_reports_bad_lengths_blocks_and_bounds():
    cache, table, L, q, up, cu = make_prefill([200, 300, 150], [20, 300, 150], 2, 16, "f16", 57)
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(torch.float16))

    def call(lens=L, tab=table, most=300, tokens=650):
        out, err = torch.full((470, 2, 128), 5.0, dtype=q.dtype, device=DEV), i32([0])
        pa.pa_latent_prefill(out, q, cu, up, cache, tab, lens, most, tokens, SCALE, device_error=err)
        return out, int(err)

    bad = L.clone()
    bad[1] = 299                                   # fewer tokens than new ones
    out, err = call(lens=bad)
    assert err == 3 and bool((out[20:320] == 5).all())
    check(out[:20], want[:20], tol[:20])
    check(out[320:], want[320:], tol[320:])
    out, err = call(most=299)
    assert err == 3 and bool((out[20:320] == 5).all())
    out, err = call(tokens=0)                      # far more tokens than the bound: the last do not fit
    assert err == 3 and bool((out[320:] == 5).all())
    check(out[:20], want[:20], tol[:20])
    cache[0] = 0
    want, tol = expect_prefill(cache, table, L, q, up, cu, 16, SCALE, eps(torch.float16))
    t = table.clone()
    t[1, 2] = 1 << 20
    out, err = call(tab=t)
    assert err == 1
    check(out[:20], want[:20], tol[:20])


def test_prefill_captured_and_replayed():
    cache, table, L, q, up, cu = make_prefill([300, 260], [200, 260], 4, 32, "bf16", 59)
    ws = torch.empty(pa.pa_latent_prefill_workspace_size(2, 4, 600), dtype=torch.uint8, device=DEV)
    out = torch.empty(460, 4, 128, dtype=torch.bfloat16, device=DEV)
    args = (out, q, cu, up, cache, table, L, 260, 600, SCALE)
    pa.pa_latent_prefill(*args, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_latent_prefill(*args, workspace=ws)
    ws.random_()
    L.copy_(i32([250, 260]))
    q.copy_(randn(gen(61), *q.shape))
    up.mul_(0.5)
    out.fill_(float("nan"))
    graph.replay()
    want, tol = expect_prefill(cache, table, L, q, up, cu, 32, SCALE, eps(torch.bfloat16))
    check(out, want, tol)


def test_serving_run_of_the_latent_calls():
    """A prompt written and prefilled in its expanded form, then a token decoded in its absorbed form: the absorbed
    result, projected, is what the expanded form gives for the same token."""
    H, bs, n = 4, 16, 150
    g = gen(67)
    table, nb, _ = tables([n], bs, 67)
    cache = torch.full((nb, bs, ROW), float("nan"), dtype=torch.float16, device=DEV)
    rows = randn(g, n, ROW).half()
    slots = (table[0].long()[:, None] * bs + torch.arange(bs, device=DEV)).flatten()[:n].contiguous()
    up = (randn(g, H, 256, LATENT) / math.sqrt(LATENT)).half()
    q = randn(g, n, H, 192).half()
    pa.pa_latent_write(rows[:-1, :LATENT], rows[:-1, LATENT:], slots[:-1], cache)
    a = run_prefill(cache, table, i32([n - 1]), q[:-1], up, i32([0, n - 1]), SCALE, n - 1, n)
    pa.pa_latent_write(rows[-1:, :LATENT], rows[-1:, LATENT:], slots[-1:], cache)
    b = run_prefill(cache, table, i32([n]), q, up, i32([0, n]), SCALE, n, n)
    want, tol = expect_prefill(cache, table, i32([n]), q, up, i32([0, n]), bs, SCALE, eps(torch.float16))
    check(a, want[:-1], tol[:-1])
    check(b, want, tol)
    absorbed = torch.cat((torch.einsum("hd,hdc->hc", q[-1, :, :128].double(), up[:, :128].double()),
                          q[-1, :, 128:].double()), -1).half()
    lat = run(cache, table, i32([n]), absorbed[None, None], SCALE)[0, 0]
    got = torch.einsum("hc,hdc->hd", lat.double(), up[:, 128:].double())
    # the absorbed query's and the latent result's roundings, through the up-projection
    x = rows_of(cache, table[0], n, bs)
    more = torch.einsum("hc,hdc->hd", eps(torch.float16) / 2 * lat.double().abs(), up[:, 128:].double().abs())
    d = (absorbed.double().abs() * eps(torch.float16) / 2) @ x.abs().T * SCALE
    spread = x[:, :LATENT].abs().amax(0) @ up[:, 128:].double().abs().transpose(1, 2)
    check(got, want[-1], tol[-1] + more + 2 * d.amax(-1)[:, None] * spread)


def test_two_streams_at_once():
    """Calls of both forms overlapping on two streams, each with its own workspace."""
    sets = []
    for i, heads in enumerate((16, 128)):
        cache, table, L, q = make([900, 2000, 70], 1, heads, 16, "bf16", 71 + i)
        want, tol = expect(cache, table, L, q, 16, SCALE, eps(torch.bfloat16))
        pc = make_prefill([400, 300], [300, 20], 4, 16, "bf16", 73 + i)
        pwant, ptol = expect_prefill(*pc, 16, SCALE, eps(torch.bfloat16))
        ws = torch.empty(pa.pa_latent_decode_workspace_size(3, 1, heads), dtype=torch.uint8, device=DEV)
        pws = torch.empty(pa.pa_latent_prefill_workspace_size(2, 4, 700), dtype=torch.uint8, device=DEV)
        out, pout = torch.empty(3, 1, heads, LATENT, dtype=q.dtype, device=DEV), torch.empty(320, 4, 128, dtype=q.dtype,
                                                                                           device=DEV)
        sets.append((torch.cuda.Stream(), cache, table, L, q, want, tol, pc, pwant, ptol, ws, pws, out, pout))
    torch.cuda.synchronize()
    for _ in range(10):
        for stream, cache, table, L, q, _, _, pc, _, _, ws, pws, out, pout in sets:
            with torch.cuda.stream(stream):
                pa.pa_latent_decode(out, q, cache, table, L, 2000, SCALE, workspace=ws)
                pcache, ptable, pL, pq, up, cu = pc
                pa.pa_latent_prefill(pout, pq, cu, up, pcache, ptable, pL, 300, 700, SCALE, workspace=pws)
    torch.cuda.synchronize()
    for _, _, _, _, _, want, tol, _, pwant, ptol, _, _, out, pout in sets:
        check(out, want, tol)
        check(pout, pwant, ptol)


def test_blocks_move_under_a_nine_head_description():
    a, b = (randn(gen(s), 6, 16, ROW).bfloat16() for s in (41, 42))
    want_a, want_b = a.clone(), b.clone()
    want_a[4], want_b[4] = a[1], b[1]
    pa.pa_copy_blocks(a.view(6, 9, 16, 64), b.view(6, 9, 16, 64), torch.tensor([[1, 4]], device=DEV))
    assert torch.equal(a, want_a) and torch.equal(b, want_b)
