"""pa_evict_tokens refuses results that lie on what it reads (CPU), and takes
tensors that lie beside each other (GPU)."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from test_eviction_abi import INVALID, PTR, evict

S, H = 3, 2                      # of the cache that `evict` describes: two heads
FAR = PTR + (1 << 16)


# (lengths that do not overlap are given overlapping weights: no case here reaches a launch)
@pytest.mark.parametrize("kw", [
    dict(sl=FAR, nl=FAR), dict(sl=FAR, nl=FAR + 4 * S - 4), dict(sl=FAR + 4 * S - 4, nl=FAR),
    dict(sl=FAR, nl=FAR + 4 * S, w=PTR, nw=PTR), dict(sl=FAR, nl=FAR + 4 * S, w=PTR, nw=PTR + 4 * S * H * 64 - 4),
    dict(sl=FAR, nl=FAR + 4 * S, w=PTR + 4 * S * H * 32 - 4, nw=PTR)])
def test_overlaps_are_refused(kw):
    kw = dict(dict(w=PTR, nw=PTR + (1 << 15)), **kw)
    assert evict(S=S, **kw) == INVALID


@pytest.mark.gpu
def test_tensors_beside_each_other_are_taken():
    from _eviction import DEV, gen, i32, randn
    k, v = (randn(gen(s), 24, H, 16, 64).half() for s in (1, 2))
    lens = i32([40, 17, 30, 0, 0, 0])
    weights = randn(gen(3), S * H * 48 + S * H * 20)
    w, nw = weights[:S * H * 48].view(S, H, 48), weights[S * H * 48:].view(S, H, 20)
    old = w.clone()
    table = torch.arange(9, dtype=torch.int32, device=DEV).view(3, 3)
    new = torch.arange(9, 15, dtype=torch.int32, device=DEV).view(3, 2)
    pa.pa_evict_tokens(k, v, table, lens[:3], w, new, lens[3:], nw, 20, 4)
    assert lens.tolist() == [40, 17, 30, 20, 17, 20] and torch.equal(w, old)
    for s, n in enumerate((40, 17, 30)):
        for h in range(H):
            kept = old[s, h, :n - 4].argsort(descending=True, stable=True)[:min(n, 20) - 4]
            kept = torch.cat((kept.sort().values, torch.arange(n - 4, n, device=DEV)))
            assert torch.equal(nw[s, h, :len(kept)], old[s, h, kept])
            rows = k[table[s].long(), h].reshape(-1, 64)[kept]
            assert torch.equal(k[new[s].long(), h].reshape(-1, 64)[:len(kept)], rows)
    with pytest.raises(pa.PaError, match="invalid argument"):
        pa.pa_evict_tokens(k, v, table, lens[:3], w, new, lens[:3], nw, 20, 4)
