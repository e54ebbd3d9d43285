"""Paged inputs and 64-bit definitions for the tests of the latent cache, of
decode weights and of token eviction."""
import math

import torch

DEV = "cuda:0"
LATENT, ROPE, ROW = 512, 64, 576
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2,
      "int8": torch.int8}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def tables(lens, bs, seed, spare=0, width=None):
    """(int32 tables [S, width], blocks in the pool, unused blocks) of sequences in blocks anywhere; entries that no
    sequence uses name no block."""
    c = torch.Generator()
    c.manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + spare + 3
    pool = torch.randperm(nb, generator=c).tolist()
    out = torch.full((len(lens), max(need + [1]) if width is None else width), -7, dtype=torch.int32)
    for s, n in enumerate(need):
        out[s, :n] = torch.tensor(pool[:n], dtype=torch.int32)
        pool = pool[n:]
    return out.to(DEV), nb, pool


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows_of(cache, table, n, bs):
    """The first n rows of a sequence in a latent cache, float64."""
    return cache[table[: -(-n // bs)].long()].reshape(-1, cache.shape[-1])[:n].double()


def head_rows(cache, table, n, bs, h):
    blocks = table[: -(-n // bs)].long()
    x = cache.view(torch.uint8)[blocks, h].view(cache.dtype)
    return x.reshape(-1, cache.shape[-1])[:n].double()


def attend(q, k, v, scale, eps):
    """softmax(scale q k^T) v in 64 bits for q [r, d], and how far a result
    may be off that rounds its weights and its outputs to a type of step eps
    and keeps sums and scores in 32 bits:
      - the output's rounding, eps / 2 of it;
      - a weight's rounding, eps / 2 of each, so eps / 2 sum w |v|;
      - a score's error d = 2^-24 (d sum |q k| scale + |x|) with d terms summed
        (at most d roundings of the partial sums) and its exponential, within
        2^-21 of it: weights off by 2 (d + 2^-21) of themselves."""
    x = q @ k.T * scale
    w = torch.softmax(x, -1)
    o = w @ v
    spread = w @ v.abs()
    size = (q.abs() @ k.abs().T).amax(-1, keepdim=True) * abs(scale)
    d = 2.0 ** -24 * (q.shape[-1] + 2) * size + 2.0 ** -21
    return o, (eps / 2) * (o.abs() + spread) * 1.01 + 2 * d * spread, w, 2 * d


def check(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got.double() - want).abs().max()), float(tol.max()))


def eps(dt):
    return torch.finfo(dt).eps


__all__ = [n for n in dir() if not n.startswith("__")]
assert math.isclose(eps(torch.bfloat16), 2.0 ** -7)
