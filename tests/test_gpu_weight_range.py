"""Many light tokens beside a heavy one: weights far below the largest of
their row, which an fp16 product still has to see."""
import pytest
import torch

import paged_kv_cache_54_gb300 as pa
from _eviction import DEV, DT, LATENT, ROW, check, eps, gen, i32, randn
from test_gpu_latent import run, run_prefill

pytestmark = pytest.mark.gpu

DROP = 17.5                          # nats between the heavy token and the others
LIGHT = float(torch.exp(torch.tensor(-DROP, dtype=torch.float64)))


def bound(n, out, top, e):
    """n light weights of 2^-25.2 of the largest.  The largest is held as at
    least 2^7 in fp16, whose smallest step's half is 2^-25: a weight is off by
    at most 2^-32 of the largest, so n of them by n 2^-32 of the values.
    Beside that each weight's and the result's half step, 2^-18 for the
    exponential, and n roundings of a total in 32 bits."""
    return n * 2.0 ** -32 * top + (e + 2.0 ** -18 + n * 2.0 ** -24) * out.abs()


def latents(L, bs, dt, seed):
    """A cache of one sequence: token 0 heavy with a latent vector of zeros, the others light, with vectors of about one."""
    nb = -(-L // bs)
    rows = torch.zeros(nb * bs, ROW, device=DEV)
    rows[1:L, :LATENT] = 1 + 0.25 * randn(gen(seed), 1, LATENT).clamp(-2, 2)
    rows[0, LATENT] = DROP
    cache = torch.empty(nb, bs, ROW, dtype=DT[dt], device=DEV)
    cache.copy_(rows.view(nb, bs, ROW))
    return cache, torch.arange(nb, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("L,S", [(250, 3), (4000, 160), (20000, 1)])
def test_latent_decode_of_many_light_tokens(L, S, heads, dt):
    cache, blocks = latents(L, 16, dt, heads)
    table = blocks.repeat(S, 1).contiguous()
    q = torch.zeros(S, 1, heads, ROW, dtype=DT[dt], device=DEV)
    q[..., LATENT] = 1
    got = run(cache, table, i32([L] * S), q, 1.0)
    v = cache.view(-1, ROW)[1, :LATENT].double()
    n = L - 1
    want = (n * LIGHT / (1 + n * LIGHT)) * v
    check(got, want.expand(S, 1, heads, LATENT), bound(n, want, v.abs(), eps(DT[dt])) + torch.finfo(DT[dt]).tiny * eps(DT[dt]))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("L", [300, 512, 9000])
def test_latent_prefill_of_many_light_tokens(L, dt):
    cache, table = latents(L, 16, dt, L)
    new, heads = 40, 2
    up = torch.zeros(heads, 256, LATENT, dtype=DT[dt], device=DEV)
    up[:, 128:] = 2.0 ** -9 * (1 + torch.arange(128, device=DEV)[:, None] % 3)      # values of about one to three
    q = torch.zeros(new, heads, 192, dtype=DT[dt], device=DEV)
    q[..., 128] = 1
    got = run_prefill(cache, table[None].contiguous(), i32([L]), q, up, i32([0, new]), 1.0, new, L)
    v = cache.view(-1, ROW)[1, :LATENT].double() @ up[0, 128:].double().T
    n = (L - new + torch.arange(new, device=DEV, dtype=torch.float64))[:, None, None]   # light tokens a row follows
    want = n * LIGHT / (1 + n * LIGHT) * v
    # (the values' rounding to fp16 on top, 2^-11 of each)
    check(got, want.expand(new, heads, 128), bound(n, want, v.abs(), eps(DT[dt]) + 2.0 ** -11) + torch.finfo(DT[dt]).tiny * eps(DT[dt]))


@pytest.mark.parametrize("qt,kt", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e5m2"), ("bf16", "int8")])
@pytest.mark.parametrize("L,S,H,D", [(128, 3, 2, 128), (2000, 80, 32, 64), (2000, 80, 32, 128)])
def test_decode_weights_of_many_light_tokens(L, S, H, D, qt, kt):
    bs, nb = 16, -(-L // 16)
    k, v = (torch.zeros(nb, H, bs, D, device=DEV) for _ in range(2))
    k[0, :, 0, 0] = 16
    v[:] = 96
    v[0, :, 0] = 0
    k, v = k.to(DT[kt]), v.to(DT[kt])
    table = torch.arange(nb, dtype=torch.int32, device=DEV).repeat(S, 1).contiguous()
    q = torch.zeros(S, H, D, dtype=DT[qt], device=DEV)
    q[..., 0] = 1
    out, w = torch.empty_like(q), torch.empty(S, H, L, device=DEV)
    err = i32([0])
    pa.pa_decode_weights(out, w, q, k, v, table, i32([L] * S), L, DROP / 16, device_error=err)
    assert int(err) == 0
    n = L - 1
    want = torch.tensor(96 * n * LIGHT / (1 + n * LIGHT), dtype=torch.float64, device=DEV)
    e = max(eps(DT[qt]), eps(torch.bfloat16 if kt == "bf16" else torch.float16))
    check(out, want.expand(S, H, D), bound(n, want, 96.0, e) + torch.finfo(DT[qt]).tiny * eps(DT[qt]))
    share = torch.full((L,), LIGHT / (1 + n * LIGHT), dtype=torch.float64, device=DEV)
    share[0] = 1 / (1 + n * LIGHT)
    check(w, share.expand(S, H, L), (2.0 ** -17 + n * 2.0 ** -24) * share)
