"""pa_decode_weights on the GPU against the definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, DT, attend, check, eps, gen, head_rows, i32, randn, tables

pytestmark = pytest.mark.gpu


def make(lens, Hq, H, D, bs, qt, kt, seed):
    g = gen(seed)
    table, nb, _ = tables(lens, bs, seed)
    wide = kt in ("f16", "bf16")
    x = randn(g, 2, nb, H, bs, D)
    x = (x * 30).round().clamp(-128, 127) if kt == "int8" else x if wide else x * 8
    x = x.to(DT[kt])
    k, v = x[0].contiguous(), x[1].contiguous()
    for s, n in enumerate(lens):   # rows behind a sequence's end hold NaN where the type has one
        if n % bs and kt != "int8":
            for c in (k, v):
                blk = c[int(table[s, n // bs])].float()
                blk[:, n % bs:] = float("nan")
                c[int(table[s, n // bs])] = blk.to(DT[kt])
    return k, v, table, i32(lens), randn(g, len(lens), Hq, D).to(DT[qt])


def expect(k, v, table, lens, q, bs, scale, ks, vs, win, decay, e, pe):
    """(out, its tolerance, weights, their tolerance); e: the output's step, pe: that of the weights' type."""
    S, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    o = torch.zeros(S, Hq, D, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    w = torch.full(win.shape, -1.0, dtype=torch.float64, device=DEV)
    wt = torch.zeros_like(w)
    ks, vs = (x if isinstance(x, torch.Tensor) else torch.full((H,), float(x), device=DEV) for x in (ks, vs))
    for s, L in enumerate(lens.tolist()):
        if L == 0:
            continue
        for h in range(H):
            kk, vv = head_rows(k, table[s], L, bs, h) * ks[h].double(), head_rows(v, table[s], L, bs, h) * vs[h].double()
            qq = q[s, h * G:(h + 1) * G].double()
            a, t, p, d = attend(qq, kk, vv, scale, max(e, pe))
            # a bf16 query against one-byte codes is rounded to fp16 (its bf16 values are fp16 values up to range)
            o[s, h * G:(h + 1) * G], tol[s, h * G:(h + 1) * G] = a, t
            w[s, h, :L] = decay * win[s, h, :L].double() + p.sum(0)
            # weights keep 32 bits: their scores' error, and a few roundings of the sum
            wt[s, h, :L] = (p * (d + 2.0 ** -20)).sum(0) + 2.0 ** -22 * w[s, h, :L].abs()
    return o, tol, w, wt


SHAPES = [
    # lens, query heads, KV heads, head_dim, block
    ([1], 4, 4, 64, 16),
    ([16, 17, 15], 8, 1, 128, 8),
    ([100, 0, 1, 63, 64, 65], 4, 2, 64, 32),
    ([700, 33], 16, 4, 128, 16),
    ([2000, 1, 500], 40, 5, 128, 16),
    ([9000], 8, 8, 128, 32),
    ([3000, 40], 2, 1, 64, 8),
    ([0], 8, 1, 128, 16),
]
TYPES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("bf16", "e5m2"), ("f16", "int8"),
         ("bf16", "int8")]


@pytest.mark.parametrize("qt,kt", TYPES)
@pytest.mark.parametrize("lens,Hq,H,D,bs", SHAPES)
def test_matches_the_definition(lens, Hq, H, D, bs, qt, kt):
    k, v, table, L, q = make(lens, Hq, H, D, bs, qt, kt, seed=Hq + D)
    ks, vs = (1.0, 1.0) if kt in ("f16", "bf16") else (0.05, 0.03)
    scale = 1.0 / math.sqrt(D)
    W = max(lens) + 5
    win = torch.rand(len(lens), H, W, generator=gen(3), device=DEV) * 4
    wout = torch.full_like(win, -1.0)
    out = torch.full_like(q, float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_decode_weights(out, wout, q, k, v, table, L, max(lens), scale, weights_in=win, decay=0.5, k_scale=ks,
                         v_scale=vs, device_error=err)
    assert int(err) == 0
    pe = eps(torch.bfloat16) if kt == "bf16" else eps(torch.float16)
    o, tol, w, wt = expect(k, v, table, L, q, bs, scale, ks, vs, win, 0.5, eps(DT[qt]), pe)
    check(out, o, tol, "out")
    check(wout, w, wt, "weights")


def test_per_head_scales_in_place_and_from_nothing():
    k, v, table, L, q = make([300, 20], 16, 4, 128, 16, "bf16", "e4m3", 5)
    ks, vs = (torch.tensor(x, device=DEV) for x in ([0.1, 0.02, 0.05, 0.03], [0.5, 0.1, 0.2, 1.0]))
    acc = torch.full((2, 4, 300), -1.0, device=DEV)
    out = torch.empty_like(q)
    pa.pa_decode_weights(out, acc, q, k, v, table, L, 300, 0.09, k_scale=ks, v_scale=vs)
    zero = torch.zeros_like(acc)
    o, tol, w, wt = expect(k, v, table, L, q, 16, 0.09, ks, vs, zero, 1.0, eps(torch.bfloat16), eps(torch.float16))
    check(out, o, tol)
    check(acc, w, wt)
    pa.pa_decode_weights(out, acc, q, k, v, table, L, 300, 0.09, weights_in=acc, decay=0.25, k_scale=ks, v_scale=vs)
    check(acc[0], 1.25 * w[0], 1.3 * wt[0] + 2.0 ** -22)
    # what a sequence's weights add up to: one a query head
    for s, n in enumerate((300, 20)):
        assert torch.allclose(acc[s, :, :n].double().sum(-1), torch.full((4,), 5.0, dtype=torch.float64, device=DEV),
                              atol=1e-4)


def test_agrees_with_plain_decode():
    lens = [(53 * s * s) % 1500 + 1 for s in range(40)]
    k, v, table, L, q = make(lens, 32, 8, 128, 16, "bf16", "bf16", 9)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode(a, q, k, v, table, L, max(lens), 0.08)
    w = torch.empty(40, 8, max(lens), device=DEV)
    pa.pa_decode_weights(b, w, q, k, v, table, L, max(lens), 0.08)
    o, tol, ww, wt = expect(k, v, table, L, q, 16, 0.08, 1.0, 1.0, torch.zeros_like(w), 1.0, eps(torch.bfloat16),
                            eps(torch.bfloat16))
    check(a, o, tol)
    check(b, o, tol)
    for s, n in enumerate(lens):
        check(w[s, :, :n], ww[s, :, :n], wt[s, :, :n])


def test_scores_of_minus_infinity_weigh_nothing():
    k, v, table, L, q = make([40], 2, 1, 64, 16, "f16", "f16", 12)
    q.fill_(1.0)
    k[table[0].long(), :, :, 0] = float("-inf")      # every token
    w, out = torch.full((1, 1, 40), 9.0, device=DEV), torch.empty_like(q)
    pa.pa_decode_weights(out, w, q, k, v, table, L, 40, 0.1)
    assert float(out.abs().sum()) == 0 and float(w.abs().sum()) == 0
    k[int(table[0, 1]), 0, 3, 0] = 0.0               # all but token 19
    pa.pa_decode_weights(out, w, q, k, v, table, L, 40, 0.1)
    assert float(w[0, 0, 19]) == 2.0 and float(w.sum()) == 2.0
    assert torch.equal(out[0], v[int(table[0, 1]), 0, 3].expand(2, 64))


def test_bad_lengths_and_blocks():
    k, v, table, L, q = make([50, 50], 8, 2, 64, 16, "f16", "f16", 14)
    w, out, err = torch.full((2, 2, 50), -1.0, device=DEV), torch.empty_like(q), i32([0])
    bad = L.clone()
    bad[0] = -3
    pa.pa_decode_weights(out, w, q, k, v, table, bad, 50, 0.1, device_error=err)
    assert int(err) == 3 and float(out[0].abs().sum()) == 0 and bool((w[0] == -1).all())
    err.zero_()
    t = table.clone()
    t[1, 1] = 10 ** 7
    k[0] = v[0] = 0
    pa.pa_decode_weights(out, w, q, k, v, t, L, 50, 0.1, device_error=err)
    assert int(err) == 1


def test_captured_and_replayed():
    k, v, table, L, q = make([500, 40, 90], 16, 2, 128, 16, "bf16", "bf16", 15)
    ws = torch.empty(pa.pa_decode_weights_workspace_size(3, 16, 2, 128, 512), dtype=torch.uint8, device=DEV)
    acc, out = torch.zeros(3, 2, 512, device=DEV), torch.empty_like(q)
    args = (out, acc, q, k, v, table, L, 512, 0.09)
    pa.pa_decode_weights(*args, weights_in=acc, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_weights(*args, weights_in=acc, workspace=ws)
    acc.zero_()
    L.copy_(i32([499, 0, 77]))
    for _ in range(3):
        graph.replay()
    assert torch.allclose(acc.sum(-1), torch.tensor([[24.0, 24], [0, 0], [24, 24]], device=DEV), atol=1e-3)
    assert float(out[1].abs().sum()) == 0


@pytest.mark.parametrize("longest", [90, 400])   # a warp a pair, and shares
def test_many_sequences_many_of_them_empty(longest):
    lens = [0 if s % 3 == 1 else (37 * s) % longest + 1 for s in range(333)]
    k, v, table, L, q = make(lens, 6, 3, 64, 8, "f16", "f16", 16)
    w, out = torch.full((333, 3, longest + 1), -1.0, device=DEV), torch.full_like(q, float("nan"))
    pa.pa_decode_weights(out, w, q, k, v, table, L, longest, 0.125)
    o, tol, ww, wt = expect(k, v, table, L, q, 8, 0.125, 1.0, 1.0, torch.zeros_like(w), 1.0, eps(torch.float16),
                            eps(torch.float16))
    check(out, o, tol, "out")
    check(w, ww, wt, "weights")


def test_past_four_gigabytes_and_weights_aligned_to_four_bytes():
    bs, H, D = 16, 8, 128
    nb = (1 << 32) // (bs * H * D * 2) + 50
    k, v = (torch.zeros(nb, H, bs, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    blocks = [nb - 1, 3, nb - 40] + list(range(nb - 30, nb - 10))
    table = i32([blocks])
    g = gen(17)
    k[table[0].long()], v[table[0].long()] = (randn(g, len(blocks), H, bs, D).bfloat16() for _ in range(2))
    L, q = i32([len(blocks) * bs - 7]), randn(g, 1, 2 * H, D).bfloat16()
    n = int(L)
    buf = torch.rand(H * (n + 2) + 1, generator=g, device=DEV)
    acc = buf[1:].view(1, H, n + 2)
    win, out = acc.clone(), torch.empty_like(q)
    pa.pa_decode_weights(out, acc, q, k, v, table, L, n, 0.09, weights_in=acc, decay=0.5)
    o, tol, w, wt = expect(k, v, table, L, q, bs, 0.09, 1.0, 1.0, win, 0.5, eps(torch.bfloat16), eps(torch.bfloat16))
    check(out, o, tol, "out")
    check(acc[:, :, :n], w[:, :, :n], wt[:, :, :n], "weights")
    assert torch.equal(acc[:, :, n:], win[:, :, n:])


def test_two_streams_at_once():
    cases = [make([1500, 40, 700], 16, 2, 128, 16, "bf16", "bf16", 18 + i) for i in range(2)]
    streams, outs = [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    for (k, v, table, L, q), st in zip(cases, streams):
        with torch.cuda.stream(st):
            w, out = torch.zeros(3, 2, 1500, device=DEV), torch.empty_like(q)
            for _ in range(4):
                pa.pa_decode_weights(out, w, q, k, v, table, L, 1500, 0.09)
            outs.append((out, w))
    torch.cuda.synchronize()
    for (k, v, table, L, q), (out, w) in zip(cases, outs):
        o, tol, ww, wt = expect(k, v, table, L, q, 16, 0.09, 1.0, 1.0, torch.zeros_like(w), 1.0, eps(torch.bfloat16),
                                eps(torch.bfloat16))
        check(out, o, tol)
        for s, n in enumerate(L.tolist()):
            check(w[s, :, :n], ww[s, :, :n], wt[s, :, :n])


@pytest.mark.parametrize("seqs", [127, 128, 129])
def test_around_the_sequences_a_warp_adds_up(seqs):
    lens = [(s * 31) % 150 if s % 4 else 0 for s in range(seqs)]
    lens[-1] = 900
    k, v, table, L, q = make(lens, 4, 2, 64, 16, "bf16", "bf16", 19)
    w, out = torch.full((seqs, 2, 900), -1.0, device=DEV), torch.full_like(q, float("nan"))
    pa.pa_decode_weights(out, w, q, k, v, table, L, 900, 0.125)
    o, tol, ww, wt = expect(k, v, table, L, q, 16, 0.125, 1.0, 1.0, torch.zeros_like(w), 1.0, eps(torch.bfloat16),
                            eps(torch.bfloat16))
    check(out, o, tol, "out")
    check(w, ww, wt, "weights")
