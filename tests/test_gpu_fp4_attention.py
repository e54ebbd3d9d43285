"""Decode and prefill over a four-bit cache on the GPU, against the plain
attention in 64 bits, with bounds counted from the kernels' roundings."""
import itertools

import numpy as np
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from tests._fp4 import DEV, Case

pytestmark = pytest.mark.gpu

EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("D,bs,G", list(itertools.product([64, 128], [8, 16, 32], [1, 2, 4, 8])))
def test_decode_every_shape(D, bs, G):
    for q, per_head in (("bf16", True), ("f16", False)):
        c = Case(D + bs + G, EDGES, G, 2, D, bs, q, per_head=per_head, width_pad=bs % 3)
        g = c.device()
        c.decode(g)
        c.check(g, f"{q}")


@pytest.mark.parametrize("P", [0, 64, 256, 1024])
@pytest.mark.parametrize("lens", [[3000], [1, 2999, 64, 0, 1025], [4097, 130], [257] * 40])
def test_decode_splits_and_joins(P, lens):
    c = Case(11, lens, 4, 3, 128, 16, "bf16", per_head=True)
    g = c.device()
    c.decode(g, P)
    c.check(g, f"P {P}")


@pytest.mark.parametrize("H,S", [(1, 1), (1, 3), (7, 2), (40, 1)])
def test_decode_odd_heads(H, S):
    c = Case(5, [700 + 13 * s for s in range(S)], 2, H, 64, 8, "f16")
    g = c.device()
    c.decode(g)
    c.check(g)


def test_decode_many_sequences():
    rng = np.random.default_rng(2)
    c = Case(6, rng.integers(0, 90, 1500).tolist(), 1, 1, 64, 16, "bf16")
    g = c.device()
    c.decode(g)
    c.check(g)


def test_decode_long_sequence_with_a_loose_length_bound():
    c = Case(8, [20011, 5], 8, 1, 128, 32, "bf16", per_head=True)
    g = c.device()
    c.decode(g, max_len=32 * g.table.shape[1])
    c.check(g)


@pytest.mark.parametrize("P", [0, 64])
@pytest.mark.parametrize("lens,G,H", [([1] * 19 + [20011], 1, 8), ([20011, 0, 5] + [600] * 17, 4, 8), ([80021], 2, 1)])
def test_decode_joins_more_pieces_than_a_round_of_the_merge(lens, G, H, P):
    # 160 pairs, the longest in over 32 pieces (one warp a head); one pair in over 512 (sixteen)
    c = Case(13, lens, G, H, 64, 32, "bf16")
    g = c.device()
    c.decode(g, P)
    c.check(g, f"P {P}")


@pytest.mark.parametrize("scale,gain", [(-0.05, 1.0), (0.0, 1.0), (0.5, 1.0), (1e-6, 3e4), (1e3, 1e-5)])
def test_decode_scales_and_query_ranges(scale, gain):
    c = Case(9, [300, 77], 8, 2, 128, 16, "bf16", scale=scale, q_gain=gain)
    g = c.device()
    c.decode(g)
    c.check(g)


def test_decode_is_deterministic_and_writes_only_its_rows():
    c = Case(12, [900, 33, 2100], 4, 4, 128, 16, "bf16")
    g = c.device()
    guard = torch.full((g.q.numel() + 512,), 5.0, dtype=g.q.dtype, device=DEV)
    g.out = guard[256:256 + g.q.numel()].view_as(g.q)
    c.decode(g)
    torch.cuda.synchronize()
    a = g.out.clone()
    for _ in range(3):
        c.decode(g)
        torch.cuda.synchronize()
        assert torch.equal(a, g.out)
    assert (guard[:256] == 5).all() and (guard[-256:] == 5).all()


def test_decode_reports_bad_blocks_and_lengths():
    c = Case(13, [100, 50], 2, 2, 64, 16, "f16")
    g = c.device()
    g.table[1, 1] = 10 ** 6
    c.decode(g)
    torch.cuda.synchronize()
    assert int(g.err.item()) == 1
    want, bound = c.plain()
    assert (np.abs(g.out[0].double().cpu().numpy() - want[0]) <= bound[0]).all()
    for bad in (-1, 10 ** 6):
        g = c.device()
        g.lens[1] = bad
        c.decode(g)
        torch.cuda.synchronize()
        assert int(g.err.item()) in (1, 3)      # the length, or a table entry behind the sequence's blocks
        assert (np.abs(g.out[0].double().cpu().numpy() - want[0]) <= bound[0]).all()


def test_decode_static_scratch_equals_decode():
    c = Case(14, [700, 64, 1], 4, 2, 128, 16, "bf16")
    g = c.device()
    c.decode(g)
    a = g.out.clone()
    out = torch.full_like(a, float("nan"))
    pa.pa_decode_static_scratch(out, g.q, g.k, g.v, g.table, g.lens, 700, c.scale, **g.kw)
    torch.cuda.synchronize()
    assert torch.equal(a, out)


PREFILL = [([5], [5]), ([1], [1]), ([300, 17, 64], [300, 1, 64]), ([700, 130, 65, 900], [33, 130, 0, 256]),
           ([129, 64, 63], [129, 64, 63])]


@pytest.mark.parametrize("D,bs,G", list(itertools.product([64, 128], [8, 16, 32], [1, 2, 4, 8])))
def test_prefill_every_shape(D, bs, G):
    for i, (lens, new) in enumerate(PREFILL[2:4]):
        c = Case(20 + i, lens, G, 2, D, bs, ("bf16", "f16")[i], new=new, per_head=bool(i), width_pad=i)
        g = c.device()
        c.prefill(g)
        c.check(g, str(lens))


@pytest.mark.parametrize("lens,new", PREFILL)
@pytest.mark.parametrize("q,gain,scale", [("bf16", 1.0, None), ("f16", 1.0, None), ("bf16", 3e4, 1e-6),
                                          ("bf16", 1e-5, 1e3), ("f16", 1.0, -0.05)])
def test_prefill_lengths_and_query_ranges(lens, new, q, gain, scale):
    c = Case(30, lens, 4, 2, 128, 16, q, new=new, q_gain=gain, scale=scale)
    g = c.device()
    c.prefill(g)
    c.check(g)


def test_prefill_of_one_token_is_the_decode():
    c = Case(31, [700, 33, 1], 4, 2, 128, 16, "bf16")
    g = c.device()
    c.prefill(g)
    c.check(g)
    c.decode(g)
    c.check(g)


def test_other_streams_and_shared_workspaces_in_two_graphs():
    a, b = Case(40, [900, 40], 4, 2, 128, 16, "bf16"), Case(41, [64, 1300], 2, 3, 128, 16, "bf16")
    ga, gb = a.device(), b.device()
    n = max(pa.pa_decode_workspace_size(2, c.G * c.H, c.H, c.D, max(c.lens)) for c in (a, b))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for c, g in ((a, ga), (b, gb)):                            # a stream given by hand
        c.decode(g, workspace=ws, stream=side)
    side.synchronize()
    a.check(ga)
    b.check(gb)
    graphs = []
    for c, g in ((a, ga), (b, gb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.decode(g, workspace=ws)
        graphs.append(graph)
    for g in (ga, gb):
        g.out.fill_(float("nan"))
    for _ in range(3):                                         # stream-ordered replays share the workspace
        for graph in graphs:
            graph.replay()
    a.check(ga)
    b.check(gb)
    gb.lens[1] = 700                                           # a replay follows new lengths
    b.lens[1] = 700
    gb.out.fill_(float("nan"))
    graphs[1].replay()
    b.check(gb)


def test_a_serving_run(tmp_path):
    """The operators together: two prompts of one prefix written, prefilled
    and decoded; one forked, its copy made; a third freed; the pool drawn
    together; every later step as if nothing had moved."""
    bs, H, G, D, nb = 16, 2, 4, 128, 64
    rng = np.random.default_rng(50)
    pool = pa.PrefixCache(nb, bs, rng.permutation(nb).tolist())
    kc = torch.full(pa.fp4_cache_shape(nb, H, bs, D), 0x7F, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, 0x7F)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(cache_dtype="fp4", k_scale=0.05, v_scale=0.05, device_error=err)
    gen = torch.Generator(device=DEV).manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV).bfloat16()  # noqa: E731
    kv = {}                                                    # (sequence, position) -> K and V rows

    def write(rows):
        slots = []
        for s, p in rows:
            kv[s, p] = randn(2, H, D)
            slots.append(pool.table(s)[p // bs] * bs + p % bs)
        x = torch.stack([kv[r] for r in rows], 1).contiguous()
        pa.pa_reshape_and_cache(x[0], x[1], torch.tensor(slots, device=DEV), kc, vc, **kw)

    lens = {}

    def outputs(seqs):
        t, n = pool.block_tables(seqs, 20)
        q = torch.stack([torch.randn(G * H, D, generator=torch.Generator().manual_seed(100 * s + int(m))).bfloat16()
                         for s, m in zip(seqs, n)]).to(DEV)
        out = torch.empty_like(q)
        table, L = torch.from_numpy(t).to(DEV), torch.from_numpy(n).to(DEV)
        pa.pa_decode(out, q, kc, vc, table, L, int(n.max()), 0.09, **kw)
        return out, q, table, L

    def check(seqs, out, q):
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for i, s in enumerate(seqs):
            rows = torch.stack([kv[s, p] for p in range(lens[s])]).double().cpu()
            for h in range(H):
                k, v = rows[:, 0, h], rows[:, 1, h]
                w = torch.softmax(0.09 * q[i, h * G:(h + 1) * G].double().cpu() @ k.T, -1)
                # four-bit K and V: near the exact rows, not equal to them
                assert float((out[i, h * G:(h + 1) * G].double().cpu() - w @ v).norm() / (w @ v).norm()) < 0.3

    shared = list(range(64))
    for s, own in ((0, 37), (1, 90), (2, 50)):
        hit = pool.add_sequence(s, shared + [1000 * (s + 1) + i for i in range(own)])
        assert hit == (0 if s == 0 else 64)
        lens[s] = 64 + own
        for p in range(hit):
            kv[s, p] = kv[0, p]
        write([(s, p) for p in range(hit, lens[s])])
    q = randn(90, G * H, D)                                    # sequence 1's own tokens over the shared blocks
    out = torch.empty_like(q)
    t, n = pool.block_tables([1], 20)
    pa.pa_prefill(out, q, torch.tensor([0, 90], dtype=torch.int32, device=DEV), kc, vc, torch.from_numpy(t).to(DEV),
                  torch.from_numpy(n).to(DEV), 90, 0.09, **kw)
    a, qa, _, _ = outputs([0, 1, 2])
    check([0, 1, 2], a, qa)
    last = torch.empty_like(q[:1])                             # its last row, as a decode
    pa.pa_decode(last, q[-1:].contiguous(), kc, vc, torch.from_numpy(t).to(DEV), torch.from_numpy(n).to(DEV), 154, 0.09,
                 **kw)
    torch.cuda.synchronize()
    assert float((last.float() - out[-1:].float()).abs().max()) <= 2.0 ** -7 * float(last.float().abs().max())
    pair = pool.fork_sequence(0, 3)
    assert pair is not None
    pa.pa_copy_blocks(kc, vc, torch.tensor([pair], dtype=torch.int64, device=DEV), cache_dtype="fp4", device_error=err)
    lens[3] = lens[0]
    for p in range(lens[0]):
        kv[3, p] = kv[0, p]
    pool.free_sequence(2)
    for step in range(20):
        for s in (0, 1, 3):
            pool.append_token(s, 7 * s + step)
        write([(s, lens[s]) for s in (0, 1, 3)])
        for s in (0, 1, 3):
            lens[s] += 1
        if step == 9:
            before, _, table, L = outputs([0, 1, 3])
            moves = pool.compact()
            assert len(moves)
            pa.pa_compact_blocks(kc, vc, torch.from_numpy(moves).to(DEV), table, L, cache_dtype="fp4",
                                 device_error=err)
            assert (table.cpu().numpy() == pool.block_tables([0, 1, 3], 20)[0]).all()
            assert max(max(pool.table(s)) for s in (0, 1, 3)) < pool.stats()["used_blocks"] + \
                pool.stats()["cached_free_blocks"]
            after, _, _, _ = outputs([0, 1, 3])
            torch.cuda.synchronize()
            assert torch.equal(before, after)                  # nothing but places has changed
    a, qa, _, _ = outputs([0, 1, 3])
    check([0, 1, 3], a, qa)


@pytest.mark.parametrize("lens", [[512], [512, 1, 0, 500] * 12, [65] * 700, [511, 64, 65, 300, 2] * 150])
def test_decode_deals_short_sequences_out_whole(lens):
    for pad in (0, 40):                                        # a looser bound on the lengths lets them be cut
        c = Case(60, lens, 2, 2, 64, 16, "bf16", per_head=True, width_pad=pad)
        g = c.device()
        c.decode(g, max_len=max(lens) + 16 * pad)
        c.check(g, f"pad {pad}")


@pytest.mark.parametrize("op", ["decode", "prefill"])
def test_a_query_of_infinities_leaves_the_others_alone(op):
    c = Case(61, [300, 70], 4, 2, 128, 16, "bf16", new=None if op == "decode" else [9, 70])
    c.q[0, 1] = float("inf")
    c.q[1, 6] = float("nan")
    c.q[0, 5] *= 1e30
    c.q[1, 2] *= 1e-30
    g = c.device()
    getattr(c, op)(g)
    torch.cuda.synchronize()
    want, bound = c.plain()
    got = g.out.double().cpu().numpy()
    rows = np.ones(got.shape[:2], bool)
    rows[0, 1] = rows[1, 6] = rows[0, 5] = False               # (scores of 1e30 leave one weight: nothing to compare)
    assert (np.abs(got - want) <= bound)[rows].all()
    assert np.isfinite(got[0, 5]).all()


def test_caches_past_four_gigabytes():
    """Blocks whose bytes lie past 2^32: written, decoded, prefilled, moved."""
    bs, H, D = 16, 8, 128
    block = H * bs * D * 9 // 16
    nb = (5 << 30) // block
    rng = np.random.default_rng(62)
    kc, vc = (torch.empty(pa.fp4_cache_shape(nb, H, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    high = (nb - 1 - rng.permutation(1000)[:20]).astype(np.int32)
    assert int(high.min()) * block > 1 << 32
    c = Case(63, [300], 4, H, D, bs, "bf16", new=[37])
    table = torch.from_numpy(high[None, :19].copy()).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(cache_dtype="fp4", k_scale=0.05, v_scale=0.05, device_error=err)
    slots = torch.tensor([int(high[p // bs]) * bs + p % bs for p in range(300)], device=DEV)
    rows = [torch.randn(300, H, D, generator=torch.Generator().manual_seed(i)).bfloat16().to(DEV) for i in range(2)]
    pa.pa_reshape_and_cache(*rows, slots, kc, vc, **kw)
    back = [torch.empty_like(r) for r in rows]
    pa.pa_gather_cache(*back, slots, kc, vc, **kw)
    # the same tokens in a small pool give the same codes, outputs and read-back
    small = [torch.empty(pa.fp4_cache_shape(19, H, bs, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    order = torch.arange(19, dtype=torch.int32, device=DEV)[None].contiguous()
    pa.pa_reshape_and_cache(*rows, torch.arange(300, device=DEV), *small, **kw)
    lens = torch.tensor([300], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 37], dtype=torch.int32, device=DEV)
    q = c.q.to(DEV)

    def outs(k, v, t):
        a, b = torch.empty_like(q[:1]), torch.empty_like(q)
        pa.pa_decode(a, q[-1:].contiguous(), k, v, t, lens, 300, 0.05, **kw)
        pa.pa_prefill(b, q, cu, k, v, t, lens, 37, 0.05, **kw)
        return a, b

    want = outs(*small, order)
    for a, b in zip(outs(kc, vc, table), want):
        assert torch.equal(a, b)
    pairs = torch.tensor(sorted((int(b), 5 + i) for i, b in enumerate(high[:19])), dtype=torch.int64, device=DEV)
    pa.pa_compact_blocks(kc, vc, pairs, table, lens, cache_dtype="fp4", device_error=err)
    for a, b in zip(outs(kc, vc, table), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and int(table.max()) < 24
    assert (back[0].float() - rows[0].float()).abs().max() < 1.0
