"""Refusals of the latent cache's calls, of pa_decode_weights and of
pa_evict_tokens: bad arguments are rejected on the host before any launch
(CPU only), and the binding rejects what the C ABI takes on trust."""
import ctypes

import pytest
import torch

import paged_kv_cache_54_gb300 as pa

PTR = 1 << 20      # aligned, never read
OK, INVALID, UNSUPPORTED = 0, 1, 2


def cache(dtype=pa.PA_BF16, bs=16, d=128, heads=2, blocks=8):
    return ctypes.byref(pa.PaCacheDesc(blocks, heads, bs, d, dtype, 1.0, 1.0, None, None))


def latent(blocks=8, bs=16, dim=512, rope=64, dtype=pa.PA_BF16):
    return ctypes.byref(pa.PaLatentDesc(blocks, bs, dim, rope, dtype))


def weights(**kw):
    a = dict(out=PTR, wout=PTR, win=None, decay=1.0, width=64, q=PTR, qt=pa.PA_BF16, S=1, Hq=4, k=PTR, v=PTR, c=cache(),
             bt=PTR, nb=4, sl=PTR, most=64, scale=0.1, ws=PTR, wb=1 << 40, err=None, st=None)
    a.update(kw)
    return pa.load_library().pa_decode_weights(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), OK), (dict(S=-1), INVALID), (dict(c=None), INVALID), (dict(out=None), INVALID),
    (dict(wout=None), INVALID), (dict(ws=None), INVALID), (dict(wb=100), INVALID), (dict(width=63), INVALID),
    (dict(q=PTR + 8), INVALID), (dict(wout=PTR + 2), INVALID), (dict(ws=PTR + 16), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(decay=float("nan")), INVALID), (dict(Hq=3), INVALID),
    (dict(Hq=6), UNSUPPORTED), (dict(Hq=32), UNSUPPORTED), (dict(c=cache(pa.PA_FP4)), UNSUPPORTED),
    (dict(c=cache(bs=64)), UNSUPPORTED), (dict(c=cache(d=96)), UNSUPPORTED), (dict(qt=pa.PA_F16), UNSUPPORTED),
    (dict(qt=pa.PA_INT8, c=cache(pa.PA_INT8)), UNSUPPORTED), (dict(most=-1), INVALID), (dict(nb=0), INVALID),
])
def test_decode_weights_refuses(kw, status):
    assert weights(**kw) == status


def evict(**kw):
    a = dict(k=PTR, v=PTR, c=cache(), bt=PTR, S=1, nb=4, sl=PTR, w=PTR, width=64, nt=PTR, nnb=2, nl=PTR, nw=PTR,
             nwidth=32, budget=32, recent=4, ws=PTR, wb=1 << 40, err=None, st=None)
    a.update(kw)
    return pa.load_library().pa_evict_tokens(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), OK), (dict(S=-1), INVALID), (dict(c=None), INVALID), (dict(budget=0), INVALID),
    (dict(recent=33), INVALID), (dict(recent=-1), INVALID), (dict(budget=33, nwidth=40), INVALID),
    (dict(nwidth=31), INVALID), (dict(w=None), INVALID), (dict(nl=None), INVALID), (dict(ws=None), INVALID),
    (dict(wb=0), INVALID), (dict(k=PTR + 8), INVALID), (dict(nt=PTR + 2), INVALID),
    (dict(c=cache(pa.PA_FP4)), UNSUPPORTED), (dict(c=cache(bs=64)), UNSUPPORTED),
    (dict(c=cache(blocks=1 << 28)), UNSUPPORTED),
])
def test_evict_refuses(kw, status):
    assert evict(**kw) == status


def write(**kw):
    a = dict(lat=PTR, rope=PTR, ls=576, rs=576, dt=pa.PA_BF16, slots=PTR, n=1, cache=PTR, d=latent(), err=None, st=None)
    a.update(kw)
    return pa.load_library().pa_latent_write(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK), (dict(n=-1), INVALID), (dict(d=None), INVALID), (dict(lat=None), INVALID),
    (dict(lat=PTR + 2), INVALID), (dict(ls=511), INVALID), (dict(rs=60), INVALID), (dict(rs=65), INVALID),
    (dict(dt=pa.PA_F16), UNSUPPORTED), (dict(d=latent(dtype=pa.PA_FP8_E4M3)), UNSUPPORTED),
    (dict(d=latent(dim=256)), UNSUPPORTED), (dict(d=latent(rope=32)), UNSUPPORTED), (dict(d=latent(bs=64)), UNSUPPORTED),
    (dict(d=latent(bs=0)), INVALID), (dict(d=latent(blocks=1 << 28)), UNSUPPORTED),
])
def test_latent_write_refuses(kw, status):
    assert write(**kw) == status


def decode(**kw):
    a = dict(out=PTR, q=PTR, qt=pa.PA_BF16, S=1, n=1, H=16, cache=PTR, d=latent(), bt=PTR, nb=4, sl=PTR, most=64,
             scale=0.1, ws=PTR, wb=1 << 40, err=None, st=None)
    a.update(kw)
    return pa.load_library().pa_latent_decode(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), OK), (dict(S=-1), INVALID), (dict(n=0), INVALID), (dict(H=0), INVALID), (dict(d=None), INVALID),
    (dict(q=None), INVALID), (dict(ws=None), INVALID), (dict(ws=PTR + 16), INVALID), (dict(wb=1000), INVALID),
    (dict(out=PTR + 8), INVALID), (dict(scale=float("nan")), INVALID), (dict(qt=pa.PA_F16), UNSUPPORTED),
    (dict(d=latent(bs=64)), UNSUPPORTED), (dict(most=-1), INVALID), (dict(n=1 << 20, H=1 << 12), UNSUPPORTED),
])
def test_latent_decode_refuses(kw, status):
    assert decode(**kw) == status


def prefill(**kw):
    a = dict(out=PTR, q=PTR, qt=pa.PA_BF16, T=8, cu=PTR, S=1, H=16, most=8, up=PTR, cache=PTR, d=latent(), bt=PTR, nb=4,
             sl=PTR, kv=64, scale=0.1, ws=PTR, wb=1 << 40, err=None, st=None)
    a.update(kw)
    return pa.load_library().pa_latent_prefill(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=0), OK), (dict(T=0), OK), (dict(most=0), OK), (dict(S=-1), INVALID), (dict(H=0), INVALID),
    (dict(kv=-1), INVALID), (dict(d=None), INVALID), (dict(up=None), INVALID), (dict(cu=None), INVALID),
    (dict(up=PTR + 8), INVALID), (dict(ws=PTR + 16), INVALID), (dict(wb=1000), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(qt=pa.PA_F16), UNSUPPORTED), (dict(S=70000), UNSUPPORTED),
    (dict(kv=1 << 27), UNSUPPORTED), (dict(d=latent(rope=128)), UNSUPPORTED),
])
def test_latent_prefill_refuses(kw, status):
    assert prefill(**kw) == status


def test_workspace_sizes():
    assert pa.pa_latent_prefill_workspace_size(2, 16, 100) >= 16 * 512 * 100
    assert pa.pa_latent_prefill_workspace_size(2, 0, 100) == 0
    assert pa.pa_latent_decode_workspace_size(4, 1, 16) > 0
    assert pa.pa_latent_decode_workspace_size(4, 0, 16) == 0
    assert pa.pa_latent_decode_workspace_size(1, 1, 128) == pa.pa_latent_decode_workspace_size(2, 1, 128)
    assert pa.pa_decode_weights_workspace_size(4, 8, 2, 128, 100) > 4 * 8 * 112 * 4
    assert pa.pa_decode_weights_workspace_size(4, 8, 3, 128, 100) == 0
    assert pa.pa_evict_workspace_size(4, 8, 100) >= 4 * 8 * 100 * 4
    assert pa.pa_evict_workspace_size(4, 8, -1) == 0


def test_binding_refuses_cpu_tensors_and_wrong_caches():
    assert pa.latent_cache_shape(4, 16) == (4, 16, 576)
    x, i = torch.zeros(2, 16, 576, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_latent_decode(x[..., :512].contiguous(), x, x, t, i, 16, 0.1)
    with pytest.raises(ValueError):
        pa.pa_latent_write(x[0, :, :512], x[0, :, 512:], torch.zeros(16, dtype=torch.int64), x)
    for shape, dt in (((4, 16, 512), torch.float16), ((4, 2, 16, 576), torch.float16), ((4, 16, 576), torch.float32)):
        with pytest.raises(ValueError):
            pa._described_latent(shape, dt)
    kc = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        pa.pa_decode_weights(kc[:, :, 0], kc, kc[:, :, 0], kc, kc, t, i, 16, 0.1)
    with pytest.raises(ValueError):
        pa.pa_evict_tokens(kc, kc, t, i, kc, t, i, kc, 4, 1)


def test_latent_decode_workspace_follows_the_gpu_not_the_rows():
    # 4 or 76 row tiles of 128 rows: the same shares, two pieces of 128 x (512 + 2) floats each
    need = 76 * 2 * 128 * 514 * 4
    for new in (1, 4, 76):
        assert need <= pa.pa_latent_decode_workspace_size(3, new, 128) <= need + 1024
    assert pa.pa_latent_decode_workspace_size(3, 152, 128) <= 2 * need + 1024
