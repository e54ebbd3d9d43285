"""pa_evict_tokens on the GPU: kept tokens, their order, their rows and
weights are exact."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, DT, gen, i32, randn, tables

pytestmark = pytest.mark.gpu


def kept(w, L, budget, recent):
    """Kept token indexes of one head, ascending (a NaN below every number)."""
    B = min(L, budget)
    r = min(recent, B)
    x = [(-float("inf") if v != v else v, v == v) for v in w[: L - r].tolist()]
    best = sorted(range(L - r), key=lambda i: (-x[i][0], not x[i][1], i))[: B - r]
    return sorted(best) + list(range(L - r, L))


def make(lens, H, D, bs, kt, budget, seed):
    g = gen(seed)
    need = [-(-min(n, budget) // bs) for n in lens]
    table, nb, free = tables(lens, bs, seed, spare=sum(need))
    k, v = ((randn(g, nb, H, bs, D) * 20).to(DT[kt]) for _ in range(2))
    new = torch.full((len(lens), max(1, -(-budget // bs))), -9, dtype=torch.int32)
    for s, n in enumerate(need):
        new[s, :n] = torch.tensor(free[:n], dtype=torch.int32)
        free = free[n:]
    return k, v, table, i32(lens), new.to(DEV)


def raw(x):
    return x.view(torch.uint8)


def run_and_check(k, v, table, L, new, w, budget, recent, bs, cache_dtype=None):
    S, H, _ = w.shape
    want_k, want_v = raw(k).clone(), raw(v).clone()
    new_w = torch.full((S, H, budget + 2), -5.0, device=DEV)
    want_w = new_w.clone()
    for s, n in enumerate(L.tolist()):
        for h in range(H):
            j = torch.tensor(kept(w[s, h].cpu(), n, budget, recent), dtype=torch.long, device=DEV)
            i = torch.arange(len(j), device=DEV)
            src, dst = table[s][j // bs].long(), new[s][i // bs].long()
            for c, o in ((want_k, k), (want_v, v)):
                c[dst, h, i % bs] = raw(o)[src, h, j % bs]
            want_w[s, h, : len(j)] = w[s, h, j]
    lens, err = torch.full((S,), -1, dtype=torch.int32, device=DEV), i32([0])
    pa.pa_evict_tokens(k, v, table, L, w, new, lens, new_w, budget, recent, cache_dtype=cache_dtype, device_error=err)
    assert int(err) == 0
    assert lens.tolist() == [min(n, budget) for n in L.tolist()]
    assert torch.equal(raw(k), want_k) and torch.equal(raw(v), want_v)
    assert torch.equal(new_w.view(torch.int32), want_w.view(torch.int32))


@pytest.mark.parametrize("kt,D,bs", [("bf16", 128, 16), ("f16", 64, 8), ("e4m3", 128, 32), ("int8", 64, 16),
                                     ("e5m2", 128, 8)])
@pytest.mark.parametrize("lens,H,budget,recent", [
    ([1], 1, 1, 0),
    ([33, 0, 7, 100], 2, 20, 5),
    ([500, 499, 64], 3, 64, 64),     # only the recent ones
    ([300], 4, 299, 0),
    ([700, 20], 8, 333, 100),
    ([2500], 2, 1025, 1),
])
def test_keeps_the_heaviest_and_the_last(lens, H, budget, recent, kt, D, bs):
    k, v, table, L, new = make(lens, H, D, bs, kt, budget, seed=budget)
    w = torch.exp(2 * randn(gen(budget + 1), len(lens), H, max(lens) + 3))
    run_and_check(k, v, table, L, new, w, budget, recent, bs)


def test_ties_zeros_and_odd_weights():
    lens, H, budget = [400, 3000], 2, 150
    k, v, table, L, new = make(lens, H, 64, 16, "f16", budget, 3)
    w = torch.zeros(2, H, 3000, device=DEV)
    w[0, 0] = torch.randint(0, 3, (3000,), generator=gen(4), device=DEV).float()   # few values
    w[0, 1, ::7] = -0.0                                                            # equal to 0
    w[1, 0] = float("nan")
    w[1, 0, 50:90] = 1.0
    w[1, 0, 90:120] = float("-inf")
    w[1, 1, 100:300] = float("inf")
    w[1, 1, 300:400] = -randn(gen(5), 100).abs()
    run_and_check(k, v, table, L, new, w, budget, 10, 16)


def test_long_sequence_and_near_keys():
    """Weights that differ only in their last bits, tokens over many steps of a block."""
    n, budget = 70001, 12345
    k, v, table, L, new = make([n], 1, 64, 32, "int8", budget, 6)
    w = (torch.full((1, 1, n), 0x3f800000, dtype=torch.int32, device=DEV)
         + torch.randint(0, 3000, (1, 1, n), generator=gen(7), device=DEV, dtype=torch.int32)).view(torch.float32)
    run_and_check(k, v, table, L, new, w, budget, 77, 32)


def test_shared_source_blocks():
    """Two sequences with one prefix are cut down to blocks of their own; the shared blocks stay as they were."""
    k, v, table, L, new = make([96, 96], 2, 128, 16, "bf16", 40, 8)
    table[1, :4] = table[0, :4]
    w = torch.rand(2, 2, 96, generator=gen(9), device=DEV)
    run_and_check(k, v, table, L, new, w, 40, 8, 16)


def test_bad_lengths_and_blocks():
    k, v, table, L, new = make([50, 60, 64], 1, 64, 16, "f16", 20, 10)
    w = torch.rand(3, 1, 64, generator=gen(11), device=DEV)
    bad = L.clone()
    bad[1] = 65
    k0 = k.clone()
    lens, new_w, err = i32([9, 9, 9]), torch.full((3, 1, 20), -1.0, device=DEV), i32([0])
    pa.pa_evict_tokens(k, v, table, bad, w, new, lens, new_w, 20, 4, device_error=err)
    assert int(err) == 3 and lens.tolist() == [20, 0, 20] and bool((new_w[1] == -1).all())
    assert torch.equal(k[new[1, 0].long()], k0[new[1, 0].long()])
    err.zero_()
    n2 = new.clone()
    n2[0, 0] = 10 ** 6
    pa.pa_evict_tokens(k, v, table, L, w, n2, lens, new_w, 20, 4, device_error=err)
    assert int(err) == 1
    err.zero_()
    t2 = table.clone()
    t2[2, 3] = -1
    pa.pa_evict_tokens(k, v, t2, L, w, new, lens, new_w, 20, 4, device_error=err)
    assert int(err) == 1


def test_decode_accumulate_evict_decode():
    """The calls as a serving loop makes them: steps that weigh the tokens, an eviction, and decoding on."""
    bs, H, G, D, L0, budget = 16, 2, 4, 64, 120, 48
    k, v, table, L, new = make([L0], H, D, bs, "f16", budget, 12)
    k.normal_(generator=gen(13)), v.normal_(generator=gen(14))
    w = torch.zeros(1, H, 128, device=DEV)
    for step in range(3):
        q = randn(gen(20 + step), 1, H * G, D).half()
        out = torch.empty_like(q)
        pa.pa_decode_weights(out, w, q, k, v, table, L, 128, 0.2, weights_in=w)
    keep = [kept(w[0, h].cpu(), L0, budget, 16) for h in range(H)]
    new_w, lens = torch.zeros(1, H, budget, device=DEV), i32([0])
    pa.pa_evict_tokens(k, v, table, L, w, new, lens, new_w, budget, 16)
    out = torch.empty_like(q)
    pa.pa_decode(out, q, k, v, new, lens, budget, 0.2)
    for h in range(H):
        j = torch.tensor(keep[h], device=DEV)
        blk = table[0][j // bs].long()
        kk, vv = k[blk, h, j % bs].double(), v[blk, h, j % bs].double()
        p = torch.softmax(q[0, h * G:(h + 1) * G].double() @ kk.T * 0.2, -1)
        assert torch.allclose(out[0, h * G:(h + 1) * G].double(), p @ vv, atol=2e-3)


def test_past_four_gigabytes_and_weights_aligned_to_four_bytes():
    bs, H, D, n, budget = 16, 8, 128, 700, 300
    nb = (1 << 32) // (bs * H * D * 2) + 200
    k, v = (torch.zeros(nb, H, bs, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    old, new = [nb - 1, 2] + list(range(nb - 60, nb - 18)), [nb - 2] + list(range(10, 28))
    table, to = i32([old]), i32([new])
    g = gen(30)
    k[table[0].long()], v[table[0].long()] = (randn(g, len(old), H, bs, D).bfloat16() for _ in range(2))
    w = torch.rand(H * (n + 1) + 1, generator=g, device=DEV)[1:].view(1, H, n + 1)
    run_and_check(k, v, table, i32([n]), to, w, budget, 20, bs)


def test_captured_and_replayed():
    k, v, table, L, new = make([300, 20, 500], 2, 64, 16, "f16", 100, 31)
    w = torch.rand(3, 2, 500, generator=gen(32), device=DEV)
    ws = torch.empty(pa.pa_evict_workspace_size(3, 2, 100), dtype=torch.uint8, device=DEV)
    lens, new_w = i32([0, 0, 0]), torch.zeros(3, 2, 100, device=DEV)
    args = (k, v, table, L, w, new, lens, new_w, 100, 10)
    pa.pa_evict_tokens(*args, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_evict_tokens(*args, workspace=ws)
    L.copy_(i32([299, 0, 433]))
    w.copy_(torch.rand(3, 2, 500, generator=gen(33), device=DEV))
    k.copy_(randn(gen(34), *k.shape)), v.copy_(randn(gen(35), *v.shape))
    before = k.clone(), v.clone()
    ws.fill_(0x7f), new_w.zero_()
    graph.replay()
    assert lens.tolist() == [100, 0, 100]
    got = k.clone(), v.clone(), new_w.clone()
    k.copy_(before[0]), v.copy_(before[1]), new_w.zero_()
    run_and_check(k, v, table, L, new, w, 100, 10, 16)     # the same from the same start, and right
    assert torch.equal(k, got[0]) and torch.equal(v, got[1])
    pa.pa_evict_tokens(k, v, table, L, w, new, lens, new_w, 100, 10)
    assert torch.equal(new_w, got[2])
