"""Values of the expanded form beside the borders between their powers of two:
sizes at which neighbouring groups of 32 tokens are stored in different units,
and groups without any value, held to the errors that independent roundings
add up to."""
import math

import pytest
import torch

from _eviction import DT, LATENT, eps, rows_of
from test_gpu_latent import SCALE, make_prefill, run_prefill

pytestmark = pytest.mark.gpu


def rms(x):
    return float(x.double().square().mean().sqrt())


def error_and_bound(cache, table, L, new, q, up, dt, got, bs):
    """(root of the mean squared error, what it may be).  Each of a row's
    terms w_i v_i carries independent relative errors: its weight's rounding
    to fp16 (2^-11), its value's (2^-11), its score's from the rounded key,
    scale e / 2 |q k| in the root of its squares; and 2^-15 covers the sums in
    32 bits and the exponential.  They add as the root of the terms' squares,
    a = sqrt(sum w^2 v^2).  Beside that a value is off by at most 2^-25 of its
    unit, a weight by 2^-25 of the largest of its row, and the result by e / 2
    of itself.  (The largest rounding stands for its mean square's root, which
    is sqrt(3) less.)"""
    e = eps(DT[dt])
    err, bound = [], []
    x = rows_of(cache, table[0], L, bs)
    hidden = torch.arange(L, device=x.device)[None] > (L - new + torch.arange(new, device=x.device))[:, None]
    for h in range(q.shape[1]):
        kv = x[:, :LATENT] @ up[h].double().T
        key, v = torch.cat((kv[:, :128], x[:, LATENT:]), 1), kv[:, 128:]
        qq = q[:, h].double()
        w = torch.softmax((qq @ key.T * SCALE).masked_fill(hidden, -math.inf), -1)
        o = w @ v
        a = (w.square() @ v.square()).sqrt()
        ds = SCALE * e / 2 * (qq.square() @ key.square().T).sqrt().amax(-1, keepdim=True)
        unit = max(1.0, float(v.abs().max()) / 2.0 ** 11)
        least = 2.0 ** -25 * (unit * w.square().sum(-1, keepdim=True).sqrt() + math.sqrt(L) * rms(v))
        err.append(got[:, h].double() - o)
        bound.append((2.0 ** -10 + 2.0 ** -15 + ds) * a + e / 2 * o.abs() + least)
    return rms(torch.stack(err)), rms(torch.stack(bound))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("L", [256, 4096])
@pytest.mark.parametrize("std", [0.0175, 0.016, 0.014, 0.03, 2.0 ** -8, 9000.0, 12000.0])
def test_values_beside_the_borders_of_their_units(std, L, dt):
    cache, table, lens, q, up, cu = make_prefill([L], [24], 2, 16, dt, seed=L + int(std * 1000))
    up[:, 128:] *= std
    got = run_prefill(cache, table, lens, q, up, cu, SCALE, 24, L)
    err, bound = error_and_bound(cache, table, L, 24, q, up, dt, got, 16)
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [[0], [3], [0, 1, 5, 7], list(range(7))])
@pytest.mark.parametrize("std", [1.0, 0.01, 2.0 ** -12])
def test_small_values_beside_groups_of_zero_rows(std, zeros, dt):
    """Rows of zeros (padding, say) take no part in the unit of a row's sums."""
    L = 256
    cache, table, lens, q, up, cu = make_prefill([L], [24], 2, 16, dt, seed=91)
    up[:, 128:] *= std
    for z in zeros:
        cache[table[0, 2 * z:2 * z + 2].long(), :, :LATENT] = 0
    got = run_prefill(cache, table, lens, q, up, cu, SCALE, 24, L)
    err, bound = error_and_bound(cache, table, L, 24, q, up, dt, got, 16)
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("L", [64, 200])
def test_sequences_of_zero_rows_alone_give_zeros(L):
    cache, table, lens, q, up, cu = make_prefill([L, 70], [L, 70], 2, 16, "bf16", seed=93)
    cache[table[0, :-(-L // 16)].long(), :, :LATENT] = 0
    got = run_prefill(cache, table, lens, q, up, cu, SCALE, max(L, 70), L + 70)
    assert not got[:L].any() and bool(torch.isfinite(got).all()) and bool(got[L:].any())


def test_the_border_lies_in_one_row():
    """One group just above 2^-4 among groups just below it, and the other way round."""
    for small, large in ((0.0624, 0.0626), (32000.0, 33000.0)):
        for odd in (0, 2, 7):
            L = 256
            cache, table, lens, q, up, cu = make_prefill([L], [24], 2, 16, "bf16", seed=95 + odd)
            up[:, 128:] *= 0.016 if small < 1 else 8500.0          # (the factors below lie near one)
            x = cache[table[0].long()].view(-1, cache.shape[-1])
            for b in range(8):   # each group's largest value where it is wanted
                part = x[32 * b:32 * b + 32, :LATENT].double()
                top = max(float((part @ up[h, 128:].double().T).abs().max()) for h in range(2))
                x[32 * b:32 * b + 32, :LATENT] = (part * (large if (b == odd) == (small < 1) else small) / top).bfloat16()
            cache[table[0].long()] = x.view(-1, 16, cache.shape[-1])
            got = run_prefill(cache, table, lens, q, up, cu, SCALE, 24, L)
            err, bound = error_and_bound(cache, table, L, 24, q, up, "bf16", got, 16)
            assert err <= bound, (small, odd, err, bound)

