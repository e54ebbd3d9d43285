"""Helpers of the four-bit cache's GPU tests: caches of random bytes, the
plain attention in 64 bits, and how far an output may be from it."""
import numpy as np
import torch

import paged_kv_cache_54_gb300 as pa
from oracle import fp4 as F4

DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}     # of the output's rounding, relative
MIN_STEP = {"f16": 2.0 ** -25, "bf16": 0.0}            # and among its subnormals, absolute


def random_cache(rng, nb, H, bs, D, top=0x47):
    """Bytes of a cache: any codes, group scales 0..top (0x40 is 2.0)."""
    tiles = rng.integers(0, 256, (nb, H, bs * D * 9 // 16), dtype=np.uint8)
    tiles[..., bs * D // 2:] = rng.integers(0, top + 1, (nb, H, bs * D // 16), dtype=np.uint8)
    return tiles.reshape(nb, H, bs, D * 9 // 16)


def poison(cache, bs, D, blocks, keep):
    """The bytes of every token that no sequence holds become NaN scales and
    large codes.  keep: {block: tokens in use}."""
    nb, H = cache.shape[:2]
    tile = cache.reshape(nb, H, -1)
    codes = tile[..., :bs * D // 2].reshape(nb, H, bs, D // 2)
    scales = tile[..., bs * D // 2:].reshape(nb, H, D // 16, bs)
    for b in range(blocks):
        codes[b, :, keep.get(b, 0):] = 0xF7
        scales[b, :, :, keep.get(b, 0):] = 0x7F
    return cache


class Case:
    """Sequences of the given lengths over a pool in shuffled order; sequence
    s's last new[s] tokens are the queries of a prefill (1 each for a decode)."""

    def __init__(self, seed, lens, G, H, D, bs, q="bf16", new=None, per_head=False, scale=None, width_pad=0,
                 q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.G, self.H, self.D, self.bs, self.qt = list(lens), G, H, D, bs, q
        need = [-(-L // bs) for L in lens]
        nb = sum(need) + 3
        order = rng.permutation(nb)
        self.table = np.full((len(lens), max(1, max(need)) + width_pad), -1, np.int32)  # unused entries: never read
        at, keep = 0, {}
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            for j, b in enumerate(order[at:at + n]):
                keep[int(b)] = min(bs, lens[s] - j * bs)
            at += n
        self.k = poison(random_cache(rng, nb, H, bs, D), bs, D, nb, keep)
        self.v = poison(random_cache(rng, nb, H, bs, D), bs, D, nb, keep)
        self.new = [1] * len(lens) if new is None else list(new)
        rows = sum(self.new)
        self.q = torch.from_numpy((rng.standard_normal((rows, H * G, D)) * q_gain).astype(np.float32)).to(DT[q])
        self.scale = 1 / np.sqrt(D) / 4 if scale is None else scale
        if per_head:
            self.ks = rng.uniform(0.2, 1.0, H).astype(np.float32)
            self.vs = rng.uniform(0.2, 3.0, H).astype(np.float32)
        else:
            self.ks = self.vs = np.ones(H, np.float32) * np.float32(0.7)
        self.per_head = per_head

    def device(self):
        g = type("G", (), {})()
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        g.k, g.v, g.table, g.q = t(self.k), t(self.v), t(self.table), self.q.to(DEV)
        g.lens = t(np.array(self.lens, np.int32))
        g.cu = t(np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32))
        g.out = torch.full_like(g.q, float("nan"))
        g.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        g.kw = dict(cache_dtype="fp4", k_scale=t(self.ks) if self.per_head else float(self.ks[0]),
                    v_scale=t(self.vs) if self.per_head else float(self.vs[0]), device_error=g.err)
        return g

    def decode(self, g, P=0, workspace=None, stream=None, max_len=None):
        return pa.pa_decode(g.out, g.q, g.k, g.v, g.table, g.lens, max(self.lens) if max_len is None else max_len,
                            self.scale, partition_size=P, workspace=workspace, stream=stream, **g.kw)

    def prefill(self, g, stream=None):
        return pa.pa_prefill(g.out, g.q, g.cu, g.k, g.v, g.table, g.lens, max(self.new), self.scale, stream=stream,
                             **g.kw)

    def plain(self):
        """(outputs, bounds), both float64 [rows, Hq, D].

        The bound counts the roundings of one output element o = sum_i w_i v_i:
        its own (half a step of its type); each weight's to fp16 (2^-11 of it,
        or 2^-25 of the largest where fp16 has no normal number: L of them);
        and the weights' changes from the scores' error, twice each (numerator
        and sum).  A score is a sum of D exact products in fp32, scaled: D + 8
        roundings, taken at 2^-23 of sum |q k|, and the exponential's own 2^-20.
        """
        with np.errstate(invalid="ignore", over="ignore"):
            return self._plain()

    def _plain(self):
        k = F4.cache_values(self.k, self.D, self.ks)
        v = F4.cache_values(self.v, self.D, self.vs)
        q = self.q.double().numpy()
        out, bound = np.zeros(q.shape), np.zeros(q.shape)
        r = 0
        for s, (L, n) in enumerate(zip(self.lens, self.new)):
            pos = np.arange(L)
            blk = self.table[s][pos // self.bs]
            for h in range(self.H):
                K, V = k[blk, h, pos % self.bs], v[blk, h, pos % self.bs]
                hs = slice(h * self.G, (h + 1) * self.G)
                for j in range(n):
                    m = L - n + j + 1
                    if m <= 0:
                        continue
                    x = q[r + j, hs]
                    sc = self.scale * (x @ K[:m].T)
                    w = np.exp(sc - sc.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    o, a = w @ V[:m], w @ np.abs(V[:m])
                    ds = (self.D + 8) * 2.0 ** -23 * abs(self.scale) * (np.abs(x) @ np.abs(K[:m]).T).max(1) + 2.0 ** -20
                    out[r + j, hs] = o
                    bound[r + j, hs] = (HALF_STEP[self.qt] * np.abs(o) + MIN_STEP[self.qt] +
                                        (2.0 ** -11 + 2 * ds[:, None]) * 1.01 * a +
                                        m * 2.0 ** -25 * np.abs(V[:m]).max())
            r += n
        return out, bound

    def check(self, g, what=""):
        torch.cuda.synchronize()
        assert int(g.err.item()) == 0, int(g.err.item())
        got = g.out.double().cpu().numpy()
        want, bound = self.plain()
        off = np.abs(got - want)
        assert np.isfinite(got).all(), what
        worst = (off / np.maximum(bound, 1e-300)).max()
        assert (off <= bound).all(), f"{what}: {worst:.3f} of the bound"
        return worst
