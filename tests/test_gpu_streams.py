"""Calls on a stream that is not the current one, with scratch of their own,
while the current stream allocates and overwrites memory of the same size."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, check, eps, gen, i32, randn
from test_gpu_latent import SCALE, expect, expect_prefill, make, make_prefill
from test_gpu_weights import expect as expect_weights
from test_gpu_weights import make as make_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_scratch_of_calls_on_another_stream_is_theirs(handle):
    b16 = torch.bfloat16
    cache, table, L, q = make([900, 2000, 70], 1, 16, 16, "bf16", 3)
    want, tol = expect(cache, table, L, q, 16, SCALE, eps(b16))
    pc, pt, pl, pq, up, cu = make_prefill([400, 300], [300, 20], 4, 16, "bf16", 5)
    pwant, ptol = expect_prefill(pc, pt, pl, pq, up, cu, 16, SCALE, eps(b16))
    k, v, wt, wl, wq = make_weights([700, 1500], 16, 4, 128, 16, "bf16", "bf16", 7)
    zero = torch.zeros(2, 4, 1500, device=DEV)
    o, otol, w, wtol = expect_weights(k, v, wt, wl, wq, 16, 0.09, 1.0, 1.0, zero, 1.0, eps(b16), eps(b16))
    blocks, el = wt[:1, :44].contiguous(), i32([700])                         # the first one's tokens, to be moved
    ek, ev = (torch.cat((c, torch.zeros_like(c[:20]))) for c in (k, v))
    new_t = torch.arange(k.shape[0], k.shape[0] + 20, dtype=torch.int32, device=DEV)[None]
    weights = randn(gen(9), 1, 4, 704)
    keep = torch.stack([torch.cat((weights[0, h, :690].argsort(descending=True, stable=True)[:290].sort().values,
                                   torch.arange(690, 700, device=DEV))) for h in range(4)])

    outs = [torch.empty_like(want, dtype=b16), torch.empty_like(pwant, dtype=b16), torch.empty_like(o, dtype=b16),
            torch.empty_like(o, dtype=b16)]
    acc, nl, nw = torch.empty_like(zero), i32([0]), torch.empty(1, 4, 300, device=DEV)
    side = torch.cuda.Stream()
    sizes = (pa.pa_latent_decode_workspace_size(3, 1, 16), pa.pa_latent_prefill_workspace_size(2, 4, 700),
             pa.pa_decode_weights_workspace_size(2, 16, 4, 128, 1500), pa.pa_evict_workspace_size(1, 4, 300),
             pa.pa_decode_workspace_size(2, 16, 4, 128, 1500))
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)          # the calls start well after the host has gone on
        kw = dict(stream=side.cuda_stream if handle else side)
        pa.pa_latent_decode(outs[0], q, cache, table, L, 2000, SCALE, **kw)
        pa.pa_latent_prefill(outs[1], pq, cu, up, pc, pt, pl, 300, 700, SCALE, **kw)
        pa.pa_decode_weights(outs[2], acc, wq, k, v, wt, wl, 1500, 0.09, **kw)
        pa.pa_evict_tokens(ek, ev, blocks, el, weights, new_t, nl, nw, 300, 10, **kw)
        pa.pa_decode(outs[3], wq, k, v, wt, wl, 1500, 0.09, **kw)
        for n in sizes * 4:                        # what an allocator that forgot the stream would hand out here
            torch.full((max(n, 256),), 0xAB, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
    check(outs[0], want, tol)
    check(outs[1], pwant, ptol)
    check(outs[2], o, otol)
    check(outs[3], o, otol)
    for s, n in enumerate((700, 1500)):
        check(acc[s, :, :n], w[s, :, :n], wtol[s, :, :n])
    assert int(nl) == 300
    for h in range(4):
        rows = k[blocks[0].long(), h].reshape(-1, 128)[keep[h]]
        assert torch.equal(ek[new_t[0].long(), h].reshape(-1, 128)[:300].view(torch.int16), rows.view(torch.int16))
        assert torch.equal(nw[0, h], weights[0, h, keep[h]])
