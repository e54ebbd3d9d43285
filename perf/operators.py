"""Cases of the four-bit paged KV cache and of page compaction, with each
operator's plain form in elementary torch operations.

Four operators, each reached through the package's public calls when ``own``
is true:

  write    new tokens' K/V rows stored in a four-bit cache through a slot
           mapping, and what the stored rows stand for read back
           (pa_reshape_and_cache, pa_gather_cache)
  decode   single-query attention over a four-bit paged cache (pa_decode)
  prefill  causal attention of several new tokens a sequence over a four-bit
           paged cache (pa_prefill)
  compact  pages moved to the front of the pool, and the block tables
           renamed to match (pa_compact_blocks)

The four-bit cache: a (block, KV head) tile holds its block_size tokens'
codes, head_dim / 2 bytes each (dimension 2j in the low half of byte j), then
one e4m3 scale for every 16 dimensions, [head_dim / 16, block_size].  A code
c (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) stands for c * its group's
scale * the KV head's scale.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
GROUP = 16


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    gqa = dict(q_heads=64, kv_heads=8, head_dim=128, block=16, q="bf16", per_head=True)
    return [
        # one decode step of a handful of sequences: latency
        dict(name="write 4 tokens", op="write", tokens=4, kv_heads=8, head_dim=128, block=16, src="bf16",
             per_head=False, padded=0.0),
        # a large batch's step with padding rows, odd count, small heads and blocks
        dict(name="write 1021 tokens d64", op="write", tokens=1021, kv_heads=12, head_dim=64, block=8, src="f16",
             per_head=True, padded=0.1),
        # prompts of many requests admitted at once
        dict(name="write 65536 tokens", op="write", tokens=65536, kv_heads=8, head_dim=128, block=16, src="bf16",
             per_head=True, padded=0.0),
        # the tiny workload's shapes: four short sequences, one query head a KV head
        dict(name="decode tiny", op="decode", seqs=4, len_lo=1, len_hi=100, log_uniform=False, q_heads=4, kv_heads=4,
             head_dim=64, block=16, q="f16", per_head=False),
        # one chat at a long context
        dict(name="decode one long", op="decode", seqs=1, len_lo=131071, len_hi=131071, log_uniform=False, **gqa),
        # the llama2-7b workload's shapes
        dict(name="decode llama2-7b", op="decode", seqs=64, len_lo=512, len_hi=4096, log_uniform=False, q_heads=32,
             kv_heads=32, head_dim=128, block=16, q="f16", per_head=False),
        # the gqa workloads' shapes: lengths over two orders of magnitude
        dict(name="decode gqa", op="decode", seqs=128, len_lo=256, len_hi=32768, log_uniform=True, **gqa),
        # the first tokens of two chats' next turns
        dict(name="prefill 2 short", op="prefill", seqs=2, new_lo=3, new_hi=17, ctx_lo=0, ctx_hi=130, q_heads=8,
             kv_heads=4, head_dim=64, block=8, q="f16", per_head=False),
        # the shared-prefix workload's shapes: suffixes after a cached prefix
        dict(name="prefill suffixes", op="prefill", seqs=128, new_lo=16, new_hi=512, ctx_lo=1024, ctx_hi=1024,
             q_heads=16, kv_heads=8, head_dim=128, block=16, q="bf16", per_head=True),
        # a long prompt in one chunk after another
        dict(name="prefill long chunk", op="prefill", seqs=1, new_lo=8191, new_hi=8191, ctx_lo=8192, ctx_hi=8192,
             q_heads=32, kv_heads=4, head_dim=128, block=32, q="bf16", per_head=False),
        # a small pool drawn together between steps
        dict(name="compact small", op="compact", blocks=96, seqs=6, fill=0.6, kv_heads=8, head_dim=64, block=16,
             cache="e4m3"),
        # a serving pool drawn together before it is shrunk
        dict(name="compact pool", op="compact", blocks=16384, seqs=200, fill=0.55, kv_heads=8, head_dim=128, block=16,
             cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "compact"])
    D, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    if op == "write":
        H = rng.choice([1, 2, 4, 5, 8, 12, 32, 40])
        return dict(op=op, tokens=_log(rng, 1, 65536 * 8 * 128 // (H * D) if H * D > 1024 else 65536), kv_heads=H,
                    head_dim=D, block=bs, src=rng.choice(["f16", "bf16"]), per_head=rng.random() < 0.5,
                    padded=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "decode":
        H, G, S = rng.choice([1, 2, 4, 5, 8, 32]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 256)
        most = min(131072, max(64, int(700_000 * 8 * 128 / (H * D * S))))  # work and padded temporaries stay bounded
        hi = _log(rng, 1, most)
        lo = rng.choice([0, 1, hi // 8, hi // 2, hi])
        return dict(op=op, seqs=S, len_lo=lo, len_hi=hi, log_uniform=lo > 0 and rng.random() < 0.5, q_heads=H * G,
                    kv_heads=H, head_dim=D, block=bs, q=rng.choice(["f16", "bf16", "bf16"]),
                    per_head=rng.random() < 0.5)
    if op == "prefill":
        H, G, S = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 128)
        most = max(2, 8192 // (S * max(1, H * G // 32)))
        new = _log(rng, 1, most)
        ctx = rng.choice([0, _log(rng, 1, most), _log(rng, 1, 2048)])
        return dict(op=op, seqs=S, new_lo=max(1, new // 4), new_hi=new, ctx_lo=ctx // 2, ctx_hi=ctx, q_heads=H * G,
                    kv_heads=H, head_dim=D, block=bs, q=rng.choice(["f16", "bf16"]), per_head=rng.random() < 0.5)
    H = rng.choice([1, 2, 4, 8])
    return dict(op=op, blocks=_log(rng, 16, 16384), seqs=_log(rng, 1, 256), fill=round(rng.uniform(0.1, 0.9), 3),
                kv_heads=H, head_dim=D, block=bs if H * D * bs <= 16384 else 16,
                cache=rng.choice(["f16", "bf16", "e4m3", "int8"]))


# --------------------------------------------------------------------------
# structure of a case (lengths are the case's; the seed orders them)
# --------------------------------------------------------------------------
def _spread(n, lo, hi, log=False):
    """n whole numbers from lo to hi at even steps (of the logarithm)."""
    if n == 1 or lo == hi:
        return np.full(n, hi, np.int64)
    t = np.linspace(0.0, 1.0, n)
    x = np.exp(np.log(lo) + t * (np.log(hi) - np.log(lo))) if log else lo + t * (hi - lo)
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def _lengths(case):
    """(total length, new tokens) of every sequence, in no order."""
    if case["op"] == "decode":
        n = _spread(case["seqs"], case["len_lo"], case["len_hi"], case["log_uniform"])
        return n, np.ones_like(n)
    new = _spread(case["seqs"], case["new_lo"], case["new_hi"])
    return _spread(case["seqs"], case["ctx_lo"], case["ctx_hi"]) + new, new


def _pages(case):
    """Live blocks of every sequence of a compaction case."""
    live = max(1, int(case["blocks"] * case["fill"]))
    n = np.full(case["seqs"], live // case["seqs"], np.int64)
    n[: live % case["seqs"]] += 1
    return n


def _moves(live, blocks):
    """(src, dst) pages that leave the live ones in blocks 0..len(live)-1, by src."""
    is_live = np.zeros(blocks, bool)
    is_live[live] = True
    n = len(live)
    src = n + np.flatnonzero(is_live[n:])
    return np.stack([src, np.flatnonzero(~is_live[:n])], 1).astype(np.int64)


def work(case):
    H, D = case["kv_heads"], case["head_dim"]
    row = H * D * 9 // 16                                 # four-bit bytes of one token's K (or V)
    if case["op"] == "write":
        n = case["tokens"] - int(case["tokens"] * case["padded"])
        return {"bytes": n * 2 * (2 * H * D + row + 2 * H * D) + 8 * case["tokens"],
                "flops": n * 2 * H * D * 8}
    if case["op"] == "compact":
        # expected moves: live blocks lie anywhere, those past the live count move
        live = int(_pages(case).sum())
        moves = live * (case["blocks"] - live) / case["blocks"]
        page = 2 * H * D * case["block"] * DTYPES[case["cache"]].itemsize
        return {"bytes": 2 * moves * page + 4 * live, "flops": 0}
    L, new = _lengths(case)
    rows = case["q_heads"] * D
    kv = int(L.sum()) * 2 * row
    if case["op"] == "decode":
        return {"bytes": kv + 2 * 2 * rows * case["seqs"], "flops": 4 * rows * int(L.sum())}
    seen = (new * (L - new) + new * (new + 1) // 2).sum()
    return {"bytes": kv + 2 * 2 * rows * int(new.sum()), "flops": 4 * rows * int(seen)}


# --------------------------------------------------------------------------
# the four-bit format, plainly
# --------------------------------------------------------------------------
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x, scale):
    """Codes (0..15) and e4m3 scales of rows x [..., H, D], head scales [H]."""
    y = x.float() / scale[:, None]
    y = y.reshape(*y.shape[:-1], -1, GROUP)
    nan = torch.isnan(y)
    y = torch.where(nan, torch.zeros_like(y), y)
    a = y.abs().amax(-1)
    s = (a / torch.full_like(a, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)  # (a division: by a number it multiplies)
    d = s.float()[..., None]
    m = torch.where(d > 0, y.abs() / d, torch.zeros_like(y))
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = code + 8 * (torch.signbit(y) & (d > 0) & ~nan)
    return code.to(torch.uint8).flatten(-2), s


def _bytes(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _split(cache, D):
    """(codes [blocks, H, bs, D/2], scales [blocks, H, D/16, bs]) views of a cache."""
    nb, H, bs, _ = cache.shape
    tile = cache.view(nb, H, -1)
    return tile[..., : bs * D // 2].view(nb, H, bs, D // 2), tile[..., bs * D // 2:].view(nb, H, D // GROUP, bs)


def _values(codes, scales, scale):
    """float32 values of codes [..., H, D/2] with group scales [..., H, D/16] (bytes), head scales [H]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    c = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (c.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2) * scale[:, None]


def _gather(cache, blocks, D, scale):
    """float32 [n, bs, H, D] of whole blocks."""
    codes, scales = _split(cache, D)
    return _values(codes[blocks].transpose(1, 2), scales[blocks].permute(0, 3, 1, 2), scale)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _head_scales(case, rng, dev):
    if not case["per_head"]:
        return 1.0, 1.0, torch.ones(case["kv_heads"], device=dev), torch.ones(case["kv_heads"], device=dev)
    k, v = (torch.from_numpy(rng.uniform(0.5, 2.0, case["kv_heads"]).astype(np.float32) / 64).to(dev)
            for _ in range(2))
    return k, v, k, v


def _rows(n, case, g, dev, outliers):
    """n rows of K (some channels several times larger, as keys have them) or V."""
    x = torch.randn(n, case["kv_heads"], case["head_dim"], generator=g, device=dev)
    if outliers:
        x *= 1.0 + 3.0 * (torch.rand(case["kv_heads"], case["head_dim"], generator=g, device=dev) > 0.95)
    return x


def _filled(blocks, case, g, dev, scale, outliers):
    """A cache of `blocks` blocks, every slot holding a quantised row."""
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    cache = torch.empty(blocks, H, bs, D * 9 // 16, dtype=torch.uint8, device=dev)
    codes, scales = _split(cache, D)
    step = max(1, (1 << 27) // (H * D * bs))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        c, s = _quantise(_rows(n * bs, case, g, dev, outliers), scale)
        codes[b:b + n] = _bytes(c).view(n, bs, H, D // 2).transpose(1, 2)
        scales[b:b + n] = s.view(torch.uint8).view(n, bs, H, D // GROUP).permute(0, 2, 3, 1)
    return cache


def prepare(case, seed):
    dev = "cuda"
    rng = np.random.Generator(np.random.PCG64(seed))
    g = torch.Generator(device=dev)
    g.manual_seed(int(rng.integers(1 << 60)))
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    st = {"case": case}
    if case["op"] == "compact":
        nb, pages = case["blocks"], _pages(case)
        order = rng.permutation(nb)
        live = order[: pages.sum()]
        table = np.zeros((case["seqs"], max(1, int(pages.max()))), np.int32)
        at = 0
        for s, n in enumerate(pages):
            table[s, :n] = live[at:at + n]
            at += n
        lens = np.where(pages > 0, (pages - 1) * bs + rng.integers(1, bs + 1, case["seqs"]), 0)
        x = torch.randn(2, nb, H, bs, D, generator=g, device=dev, dtype=torch.float16)
        if case["cache"] == "int8":
            x = (x * 32).round()
        x = x.to(DTYPES[case["cache"]])
        st.update(k=x[0].contiguous(), v=x[1].contiguous(), table=torch.from_numpy(table).to(dev),
                  lens=torch.from_numpy(lens.astype(np.int32)).to(dev),
                  pairs=torch.from_numpy(_moves(live, nb)).to(dev),
                  err=torch.zeros(1, dtype=torch.int32, device=dev))
        return st
    ka, va, ks, vs = _head_scales(case, rng, dev)
    st.update(k_scale=ka, v_scale=va, ks=ks, vs=vs, err=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "write":
        n = case["tokens"]
        nb = -(-n * 5 // (4 * bs)) + 1
        slots = rng.permutation(nb)[: -(-n // bs)][:, None] * bs + np.arange(bs)  # whole blocks in turn, as prompts
        slots = slots.reshape(-1)[:n].copy()
        slots[rng.permutation(n)[: int(n * case["padded"])]] = -1
        dt = DTYPES[case["src"]]
        st.update(key=_rows(n, case, g, dev, True).to(dt), value=_rows(n, case, g, dev, False).to(dt),
                  slots=torch.from_numpy(slots).to(dev), real=torch.from_numpy(np.flatnonzero(slots >= 0)).to(dev),
                  k=torch.zeros(nb, H, bs, D * 9 // 16, dtype=torch.uint8, device=dev),
                  v=torch.zeros(nb, H, bs, D * 9 // 16, dtype=torch.uint8, device=dev),
                  k_out=torch.empty(n, H, D, dtype=dt, device=dev), v_out=torch.empty(n, H, D, dtype=dt, device=dev))
        return st
    L, new = _lengths(case)
    mix = rng.permutation(len(L))
    L, new = L[mix], new[mix]
    need = -(-L // bs)
    nb = max(1, int(need.sum() * 5 // 4))
    pool = rng.permutation(nb)
    table = np.zeros((len(L), max(1, int(need.max()))), np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = pool[at:at + n]
        at += n
    rows = len(L) if case["op"] == "decode" else int(new.sum())
    q = torch.randn(rows, case["q_heads"], D, generator=g, device=dev).to(DTYPES[case["q"]])
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(L)), new)  # a prefill's query rows: their sequence, and place among its new tokens
    st.update(seq=torch.from_numpy(seq).to(dev), place=torch.from_numpy(np.arange(len(seq)) - cu[seq]).to(dev))
    st.update(k=_filled(nb, case, g, dev, ks, True), v=_filled(nb, case, g, dev, vs, False), q=q,
              out=torch.empty_like(q), table=torch.from_numpy(table).to(dev),
              lens=torch.from_numpy(L.astype(np.int32)).to(dev), cu=torch.from_numpy(cu).to(dev),
              max_len=int(L.max()), max_new=int(new.max()), scale=1.0 / math.sqrt(D))
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    return {"write": _write, "decode": _decode, "prefill": _prefill, "compact": _compact}[st["case"]["op"]](st)


def _write(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        how = dict(cache_dtype="fp4", k_scale=st["k_scale"], v_scale=st["v_scale"], device_error=st["err"])
        pa.pa_reshape_and_cache(st["key"], st["value"], st["slots"], st["k"], st["v"], **how)
        pa.pa_gather_cache(st["k_out"], st["v_out"], st["slots"], st["k"], st["v"], **how)
        return st["k_out"], st["v_out"]
    return _store(st, "key", "k", st["ks"]), _store(st, "value", "v", st["vs"])


def _store(st, rows, cache, scale):
    D, bs = st["case"]["head_dim"], st["case"]["block"]
    real = st["real"]
    at = st["slots"][real]
    blk, off = at // bs, at % bs
    codes, scales = _split(st[cache], D)
    c, s = _quantise(st[rows][real], scale)
    codes[blk, :, off] = _bytes(c)
    scales[blk, :, :, off] = s.view(torch.uint8)
    out = torch.zeros_like(st[rows])
    out[real] = _values(codes[blk, :, off], scales[blk, :, :, off], scale).to(out.dtype)
    return out


def _decode(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        if "workspace" not in st:
            S, Hq, D = st["q"].shape
            n = pa.pa_decode_workspace_size(S, Hq, st["case"]["kv_heads"], D, st["max_len"])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device=st["q"].device)
        return pa.pa_decode(st["out"], st["q"], st["k"], st["v"], st["table"], st["lens"], st["max_len"], st["scale"],
                            cache_dtype="fp4", k_scale=st["k_scale"], v_scale=st["v_scale"],
                            workspace=st["workspace"], device_error=st["err"])
    S, Hq, D = st["q"].shape
    H = st["case"]["kv_heads"]
    # every sequence at the longest one's length: [S, H, Lmax, D]
    k, v = (_gather(st[c], st["table"].long().flatten(), D, st[s]).view(S, -1, H, D).transpose(1, 2)
            for c, s in (("k", "ks"), ("v", "vs")))
    score = torch.matmul(st["q"].float().view(S, H, -1, D) * st["scale"], k.transpose(2, 3))
    seen = torch.arange(k.shape[2], device=k.device) < st["lens"][:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(S, Hq, D).to(st["q"].dtype)


def _prefill(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        return pa.pa_prefill(st["out"], st["q"], st["cu"], st["k"], st["v"], st["table"], st["lens"], st["max_new"],
                             st["scale"], cache_dtype="fp4", k_scale=st["k_scale"], v_scale=st["v_scale"],
                             device_error=st["err"])
    T, Hq, D = st["q"].shape
    H, S, n = st["case"]["kv_heads"], st["lens"].numel(), st["max_new"]
    k, v = (_gather(st[c], st["table"].long().flatten(), D, st[s]).view(S, -1, H, D).transpose(1, 2)
            for c, s in (("k", "ks"), ("v", "vs")))
    # every sequence with as many query rows as the one with most: [S, H, G, n, D]
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    j = torch.arange(n, device=k.device)
    row = st["cu"][:-1].long()[:, None] + j
    q = st["q"][row.clamp(max=T - 1)].float().view(S, n, H, -1, D).permute(0, 2, 3, 1, 4) * st["scale"]
    pos = (st["lens"].long() - new)[:, None] + j
    seen = torch.arange(k.shape[2], device=k.device) <= pos[..., None]
    score = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (-1, n))
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, n)) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4)[st["seq"], st["place"]].reshape(T, Hq, D).to(st["q"].dtype)


def _compact(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        pa.pa_compact_blocks(st["k"], st["v"], st["pairs"], st["table"], st["lens"], cache_dtype=st["case"]["cache"],
                             device_error=st["err"])
        return st["k"], st["v"], st["table"]
    src, dst = st["pairs"][:, 0], st["pairs"][:, 1]
    st["k"].view(torch.uint8)[dst] = st["k"].view(torch.uint8)[src]
    st["v"].view(torch.uint8)[dst] = st["v"].view(torch.uint8)[src]
    name = torch.arange(st["k"].shape[0], dtype=torch.int32, device=src.device)
    name[src] = dst.int()
    used = torch.arange(st["table"].shape[1], device=src.device) * st["case"]["block"] < st["lens"][:, None]
    st["table"].copy_(torch.where(used, name[st["table"].long()], st["table"]))
    return st["k"], st["v"], st["table"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _pow2(e):
    """2^e for whole numbers e from -32 to 31."""
    return torch.tensor([2.0 ** k for k in range(-32, 32)], dtype=torch.float64, device=e.device)[e.long() + 32]


def _exact_stored(x, scale):
    """What rows x [n, H, D] stand for once stored: every rounding of the format, each on 64-bit numbers."""
    y = (x.double() / scale.double()[None, :, None]).float().double()
    y = torch.nan_to_num(y, nan=0.0, posinf=math.inf, neginf=-math.inf)
    n, H, D = y.shape
    y = y.view(n, H, D // GROUP, GROUP)
    a = y.abs().max(-1, keepdim=True).values
    a = a / torch.full_like(a, 6.0)
    # e4m3: steps of 2^(e-3) in the binade of 2^e, from e = -6 on; 448 at most
    e = (torch.frexp(a.clamp(min=2.0 ** -40)).exponent - 1).clamp(min=-6)
    step = _pow2(e - 3)
    s = (torch.round(a / step) * step).clamp(max=448.0)
    r = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    # e2m1: steps of 2^(e-1) from e = 0 on; 6 at most
    e = (torch.frexp(r.abs().clamp(min=0.5, max=8.0)).exponent - 1).clamp(0, 2)
    step = _pow2(e - 1)
    r = (torch.round(r / step) * step).clamp(-6.0, 6.0)
    return (r * s).view(n, H, D) * scale.double()[None, :, None]


def _exact_tile(cache, blocks, D):
    """float64 [n * bs, H, D] of blocks, before the head's scale, from the bits."""
    nb, H, bs, w = cache.shape
    t = cache[blocks].view(len(blocks), H, bs * w).long()
    c = t[..., : bs * D // 2].view(-1, H, bs, D // 2)
    c = torch.cat((c[..., None] % 16, c[..., None] // 16), -1).view(-1, H, bs, D)
    ce, cm = (c // 2) % 4, (c % 2).double()
    mag = torch.where(ce > 0, (1 + cm / 2) * _pow2(ce - 1), cm / 2)
    c = torch.where(c >= 8, -mag, mag)
    s = t[..., bs * D // 2:].view(-1, H, D // GROUP, bs)
    se, sm = (s // 8) % 16, (s % 8).double()
    s = torch.where(se > 0, (1 + sm / 8) * _pow2(se - 7), sm * 2.0 ** -9)
    s = s.permute(0, 1, 3, 2).repeat_interleave(GROUP, -1)
    return (c * s).permute(0, 2, 1, 3).reshape(-1, H, D)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        out = []
        for rows, scale in (("key", "ks"), ("value", "vs")):
            x = torch.zeros(st[rows].shape, dtype=torch.float64, device="cuda")
            real = st["real"]
            x[real] = _exact_stored(st[rows][real], st[scale])
            out.append(x)
        return tuple(out)
    if case["op"] == "compact":
        k, v = st["k"].clone(), st["v"].clone()
        for src, dst in st["pairs"].tolist():
            k[dst], v[dst] = st["k"][src], st["v"][src]
        name = dict(st["pairs"].tolist())
        t = [[name.get(b, b) if j * case["block"] < n else b for j, b in enumerate(row)]
             for row, n in zip(st["table"].tolist(), st["lens"].tolist())]
        return (k.double() if k.is_floating_point() else k, v.double() if v.is_floating_point() else v,
                torch.tensor(t, dtype=torch.int32, device="cuda"))
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    if case["op"] == "decode":
        cu = list(range(len(lens) + 1))
    G = case["q_heads"] // H
    for s, n in enumerate(lens):
        if n == 0:
            continue
        blocks = st["table"][s, : -(-n // bs)].long()
        k = _exact_tile(st["k"], blocks, D)[:n] * st["ks"].double()[None, :, None]
        v = _exact_tile(st["v"], blocks, D)[:n] * st["vs"].double()[None, :, None]
        q = st["q"][cu[s]:cu[s + 1]].double()
        m = len(q)
        for r in range(0, m, 2048):
            x = q[r:r + 2048]
            pos = n - m + r + torch.arange(len(x), device="cuda")
            hidden = torch.arange(n, device="cuda")[None] > pos[:, None]
            for h in range(H):
                w = torch.einsum("igd,jd->gij", x[:, h * G:(h + 1) * G], k[:, h]) / math.sqrt(D)
                w = torch.softmax(w.masked_fill_(hidden, -math.inf), -1)
                out[cu[s] + r:cu[s] + r + len(x), h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", w, v[:, h])
    return out
