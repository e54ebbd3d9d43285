"""Cases of the latent (shared-vector) paged cache with its attention, and of
eviction by accumulated attention weight, with each operator's plain form in
elementary torch operations.

Five operators, each reached through the package's public calls when ``own``
is true:

  latent_write    new tokens' latent and rotary rows stored through a slot
                  mapping (pa_latent_write)
  latent_decode   absorbed attention of one or a few new tokens a sequence
                  over the latent cache (pa_latent_decode)
  latent_prefill  expanded causal attention of a chunk of new tokens over the
                  latent cache (pa_latent_prefill)
  weights         single-query decode attention that also adds every token's
                  attention weight to an accumulator (pa_decode_weights)
  evict           each head's tokens of largest accumulated weight, and the
                  most recent ones, moved to new blocks (pa_evict_tokens)

The latent cache [num_blocks, block_size, 576] holds a token's latent vector
(512) and its rotary key (64), shared by all heads.  Absorbed: queries of 576
against the rows themselves, weighted sums of their first 512.  Expanded: head
h's key is (up[h, :128] latent, rotary), its value up[h, 128:] latent.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
ROW = LATENT + ROPE


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a handful of sequences: latency
        dict(name="latent write 5 tokens", op="latent_write", tokens=5, block=16, dtype="bf16", padded=0.0),
        # prompts of many requests admitted at once, some rows padding
        dict(name="latent write 32768 tokens", op="latent_write", tokens=32768, block=16, dtype="bf16", padded=0.05),
        # four short chats, the heads of one device out of eight
        dict(name="latent decode tiny", op="latent_decode", seqs=4, new=1, len_lo=1, len_hi=100, log_uniform=False,
             heads=16, block=16, dtype="f16"),
        # one chat at a long context, with a draft token to verify
        dict(name="latent decode one long", op="latent_decode", seqs=1, new=2, len_lo=131071, len_hi=131071,
             log_uniform=False, heads=16, block=32, dtype="bf16"),
        # a serving batch with all heads on one device
        dict(name="latent decode batch", op="latent_decode", seqs=128, new=1, len_lo=512, len_hi=4096,
             log_uniform=False, heads=128, block=16, dtype="bf16"),
        # the first tokens of two chats' next turns
        dict(name="latent prefill 2 short", op="latent_prefill", seqs=2, new_lo=3, new_hi=17, ctx_lo=0, ctx_hi=130,
             heads=16, block=8, dtype="f16"),
        # suffixes after a cached prefix
        dict(name="latent prefill suffixes", op="latent_prefill", seqs=32, new_lo=16, new_hi=512, ctx_lo=1024,
             ctx_hi=1024, heads=16, block=16, dtype="bf16"),
        # a long prompt in one chunk after another
        dict(name="latent prefill long chunk", op="latent_prefill", seqs=1, new_lo=4095, new_hi=4095, ctx_lo=4096,
             ctx_hi=4096, heads=64, block=32, dtype="bf16"),
        # a small batch whose weights are kept
        dict(name="weights tiny", op="weights", seqs=4, len_lo=1, len_hi=100, log_uniform=False, q_heads=4,
             kv_heads=4, head_dim=64, block=16, q="f16", cache="f16"),
        # the gqa workloads' shapes: lengths over two orders of magnitude
        dict(name="weights gqa", op="weights", seqs=64, len_lo=256, len_hi=32768, log_uniform=True, q_heads=64,
             kv_heads=8, head_dim=128, block=16, q="bf16", cache="bf16"),
        # one chat brought back to its budget
        dict(name="evict one", op="evict", seqs=1, len_lo=1237, len_hi=1237, budget=1000, recent=128, kv_heads=8,
             head_dim=128, block=16, cache="bf16"),
        # a batch of long chats cut to a quarter
        dict(name="evict batch", op="evict", seqs=32, len_lo=4096, len_hi=16384, budget=4096, recent=512, kv_heads=8,
             head_dim=128, block=16, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["latent_write", "latent_decode", "latent_decode", "latent_prefill", "latent_prefill", "weights",
                     "evict"])
    bs, dt = rng.choice([8, 16, 32]), rng.choice(["f16", "bf16"])
    if op == "latent_write":
        return dict(op=op, tokens=_log(rng, 1, 32768), block=bs, dtype=dt, padded=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "latent_decode":
        S, H, new = _log(rng, 1, 256), rng.choice([1, 5, 8, 16, 16, 20, 32, 64, 128, 128]), rng.choice([1, 1, 1, 2, 3, 4])
        # the work and the plain form's padded temporaries stay bounded
        hi = _log(rng, 1, min(131072, max(64, 320_000 // S, 64)) // max(1, new * H // 128))
        lo = rng.choice([0, 1, hi // 8, hi // 2, hi])
        return dict(op=op, seqs=S, new=new, len_lo=min(hi, max(lo, 0)), len_hi=hi,
                    log_uniform=lo > 0 and rng.random() < 0.5, heads=H, block=bs, dtype=dt)
    if op == "latent_prefill":
        S, H = _log(rng, 1, 64), rng.choice([1, 4, 8, 16, 16, 32, 64, 128])
        new = _log(rng, 1, min(4096, max(2, int(math.sqrt(4096 * 8191 * 64 / (S * H * 4))))))
        ctx = rng.choice([0, _log(rng, 1, new), _log(rng, 1, max(1, min(4096, 60_000 * 16 // (S * H))))])
        ctx = min(ctx, max(1, 4096 * 8191 * 64 // (S * H * new) - new))
        return dict(op=op, seqs=S, new_lo=max(1, new // 4), new_hi=new, ctx_lo=ctx // 2, ctx_hi=ctx, heads=H, block=bs,
                    dtype=dt)
    D = rng.choice([64, 128])
    cache = rng.choice([dt, dt, "e4m3", "int8"])
    if op == "weights":
        H, G, S = rng.choice([1, 2, 4, 5, 8, 32]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 256)
        hi = _log(rng, 1, min(131072, max(64, int(400_000 * 8 * 128 / (H * D * S)))))
        lo = rng.choice([0, 1, hi // 8, hi // 2, hi])
        return dict(op=op, seqs=S, len_lo=lo, len_hi=hi, log_uniform=lo > 0 and rng.random() < 0.5, q_heads=H * G,
                    kv_heads=H, head_dim=D, block=bs, q=dt, cache=cache)
    H, S = rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
    hi = _log(rng, 16, min(65536, max(64, 500_000 * 8 // (H * S))))
    budget = max(1, int(hi * rng.choice([0.1, 0.25, 0.5, 0.9])))
    return dict(op=op, seqs=S, len_lo=rng.choice([1, hi // 2, hi]), len_hi=hi, budget=budget,
                recent=rng.choice([0, budget // 8, budget // 2]), kv_heads=H, head_dim=D, block=bs, cache=cache)


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
    if case["op"] == "latent_prefill":
        new = _spread(case["seqs"], case["new_lo"], case["new_hi"])
        return _spread(case["seqs"], case["ctx_lo"], case["ctx_hi"]) + new, new
    L = _spread(case["seqs"], case["len_lo"], case["len_hi"], case.get("log_uniform", False))
    return L, np.full_like(L, case.get("new", 1))


def work(case):
    op = case["op"]
    if op == "latent_write":
        n = case["tokens"] - int(case["tokens"] * case["padded"])
        return {"bytes": n * 2 * 2 * ROW + 8 * case["tokens"], "flops": 0}
    L, new = _lengths(case)
    total = int(L.sum())
    if op == "latent_decode":
        rows = case["seqs"] * case["new"] * case["heads"]
        # the tokens that each new token's heads see (none before the first)
        seen = sum(int(np.maximum(L - j, 0).sum()) for j in range(case["new"])) * case["heads"]
        return {"bytes": total * 2 * ROW + rows * 2 * (ROW + LATENT), "flops": seen * 2 * (ROW + LATENT)}
    if op == "latent_prefill":
        H = case["heads"]
        seen = new * (L - new) + new * (new + 1) // 2
        # the cheaper form of each sequence: keys and values expanded, or queries and outputs absorbed
        expanded = 2 * L * LATENT * (NOPE + VALUE) + seen * 2 * (NOPE + ROPE + VALUE)
        absorbed = 2 * new * LATENT * (NOPE + VALUE) + seen * 2 * (ROW + LATENT)
        return {"bytes": total * 2 * ROW + H * 2 * (NOPE + VALUE) * LATENT
                + int(new.sum()) * H * 2 * (NOPE + ROPE + VALUE),
                "flops": int(np.minimum(expanded, absorbed).sum()) * H}
    H, D = case["kv_heads"], case["head_dim"]
    row = H * D * DTYPES[case["cache"]].itemsize
    if op == "weights":
        q = case["q_heads"] * D
        return {"bytes": total * (2 * row + 2 * 4 * H) + 2 * 2 * q * case["seqs"], "flops": 4 * q * total}
    kept = int(np.minimum(L, case["budget"]).sum())
    return {"bytes": kept * 2 * 2 * row + 4 * H * (total + kept), "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(need, rng, spare=0):
    """(block tables [S, widest], number of blocks, unused blocks) of sequences in blocks anywhere in a pool."""
    nb = max(1, int(need.sum() * 5 // 4)) + spare
    pool = rng.permutation(nb)
    table = np.zeros((len(need), max(1, int(need.max()))), np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = pool[at:at + n]
        at += n
    return table, nb, pool[at:]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _latent_rows(n, g, dt):
    """Latent rows as a norm with a learned weight leaves them, some channels larger, and rotary keys."""
    w = 0.5 + torch.rand(LATENT, generator=g, device="cuda")
    w *= 1.0 + 3.0 * (torch.rand(LATENT, generator=g, device="cuda") > 0.98)
    return (_randn(g, n, LATENT) * w).to(dt), _randn(g, n, ROPE).to(dt)


def _stored(x, cache):
    """Rows as a cache of the given type holds them, and their scale."""
    if cache == "int8":
        return (x * 32).round().clamp(-128, 127).to(torch.int8), 1.0 / 32
    if cache == "e4m3":
        return (x * 16).to(torch.float8_e4m3fn), 1.0 / 16
    return x.to(DTYPES[cache]), 1.0


def prepare(case, seed):
    dev, op, bs = "cuda", case["op"], case["block"]
    rng = np.random.Generator(np.random.PCG64(seed))
    g = torch.Generator(device=dev)
    g.manual_seed(int(rng.integers(1 << 60)))

    def dev_of(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    st = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    if op == "latent_write":
        n, dt = case["tokens"], DTYPES[case["dtype"]]
        nb = -(-n * 5 // (4 * bs)) + 1
        slots = rng.permutation(nb)[: -(-n // bs)][:, None] * bs + np.arange(bs)  # whole blocks in turn, as prompts
        slots = slots.reshape(-1)[:n].copy()
        slots[rng.permutation(n)[: int(n * case["padded"])]] = -1
        # both parts are views of the down-projection's output
        both = torch.cat(_latent_rows(n, g, dt), 1)
        st.update(latent=both[:, :LATENT], rope=both[:, LATENT:], slots=dev_of(slots),
                  real=dev_of(np.flatnonzero(slots >= 0)), cache=torch.zeros(nb, bs, ROW, dtype=dt, device=dev))
        return st
    L, new = _lengths(case)
    mix = rng.permutation(len(L))
    L, new = L[mix], new[mix]
    S = len(L)
    st.update(lens=dev_of(L.astype(np.int32)), max_len=int(L.max()))
    if op in ("latent_decode", "latent_prefill"):
        dt, H = DTYPES[case["dtype"]], case["heads"]
        table, nb, _ = _tables(-(-L // bs), rng)
        latent, rope = _latent_rows(nb * bs, g, dt)
        st.update(table=dev_of(table), cache=torch.cat((latent, rope), 1).view(nb, bs, ROW),
                  scale=1.0 / math.sqrt(NOPE + ROPE))
        if op == "latent_decode":
            # a query absorbed through the keys' up-projection: its latent part is smaller than its rotary one
            q = torch.cat((0.4 * _randn(g, S, case["new"], H, LATENT), _randn(g, S, case["new"], H, ROPE)), -1)
            st.update(q=q.to(dt), out=torch.empty(S, case["new"], H, LATENT, dtype=dt, device=dev))
            return st
        T = int(new.sum())
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        seq = np.repeat(np.arange(S), new)
        st.update(q=_randn(g, T, H, NOPE + ROPE).to(dt), out=torch.empty(T, H, VALUE, dtype=dt, device=dev),
                  up=(_randn(g, H, NOPE + VALUE, LATENT) / math.sqrt(LATENT)).to(dt), cu=dev_of(cu), seq=dev_of(seq),
                  place=dev_of(np.arange(T) - cu[seq]), max_new=int(new.max()), tokens=int(L.sum()))
        return st
    H, D = case["kv_heads"], case["head_dim"]
    kept = np.minimum(L, case.get("budget", 0))
    table, nb, free = _tables(-(-L // bs), rng, spare=int((-(-kept // bs)).sum()))
    k, ks = _stored(_randn(g, nb, H, bs, D) * (1.0 + 3.0 * (_randn(g, H, 1, D) > 1.6)), case["cache"])
    v, vs = _stored(_randn(g, nb, H, bs, D), case["cache"])
    # weights so far: a few heavy tokens, many light ones, some that were never seen
    w = torch.exp(2.0 * _randn(g, S, H, st["max_len"])) * (torch.rand(S, H, st["max_len"], generator=g, device=dev) > 0.05)
    st.update(table=dev_of(table), k=k, v=v, ks=ks, vs=vs, weights=w)
    if op == "weights":
        st.update(q=_randn(g, S, case["q_heads"], D).to(DTYPES[case["q"]]), scale=1.0 / math.sqrt(D),
                  new_weights=torch.zeros_like(w))
        st["out"] = torch.empty_like(st["q"])
        return st
    new_table = np.zeros((S, max(1, -(-case["budget"] // bs))), np.int32)
    at = 0
    for s, n in enumerate(-(-kept // bs)):
        new_table[s, :n] = free[at:at + n]
        at += n
    st.update(new_table=dev_of(new_table), new_lens=torch.zeros(S, dtype=torch.int32, device=dev),
              new_weights=torch.zeros(S, H, case["budget"], device=dev))
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    return {"latent_write": _latent_write, "latent_decode": _latent_decode, "latent_prefill": _latent_prefill,
            "weights": _weights, "evict": _evict}[st["case"]["op"]](st)


def _workspace(st, size):
    """The call's scratch, sized and allocated once for its shapes."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _latent_write(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        pa.pa_latent_write(st["latent"], st["rope"], st["slots"], st["cache"], device_error=st["err"])
        return st["cache"]
    real = st["real"]
    at = st["slots"][real]
    rows = st["cache"].view(-1, ROW)
    rows[at, :LATENT] = st["latent"][real]
    rows[at, LATENT:] = st["rope"][real]
    return st["cache"]


def _rows(st):
    """float32 [S, longest in whole blocks, 576] rows of every sequence, zero behind its end."""
    x = st["cache"][st["table"].long()].flatten(1, 2).float()
    here = torch.arange(x.shape[1], device=x.device) < st["lens"][:, None]
    return torch.where(here[..., None], x, 0.0)


def _softmax_(score, seen):
    """exp(score - largest) where seen, in place, and 1 / sum (0 where nothing is seen)."""
    score.masked_fill_(~seen, -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, 1.0 / total, 0.0)


def _latent_decode(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        S, n, H, _ = st["q"].shape
        return pa.pa_latent_decode(st["out"], st["q"], st["cache"], st["table"], st["lens"], st["max_len"], st["scale"],
                                   workspace=_workspace(st, lambda: pa.pa_latent_decode_workspace_size(S, n, H)),
                                   device_error=st["err"])
    x = _rows(st)
    S, n, H, _ = st["q"].shape
    score = torch.matmul(st["q"].float().flatten(1, 2) * st["scale"], x.transpose(1, 2)).view(S, n, H, -1)
    # new token j of n sees the sequence's tokens but the last n - 1 - j
    last = st["lens"][:, None] - n + torch.arange(1, n + 1, device=x.device)
    seen = torch.arange(x.shape[1], device=x.device) < last[:, :, None, None]
    p, inv = _softmax_(score, seen)
    o = torch.matmul(p.flatten(1, 2), x[..., :LATENT]).view(S, n, H, LATENT) * inv
    return o.to(st["q"].dtype)


def _latent_prefill(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        H = st["case"]["heads"]
        space = _workspace(st, lambda: pa.pa_latent_prefill_workspace_size(len(st["lens"]), H, st["tokens"]))
        return pa.pa_latent_prefill(st["out"], st["q"], st["cu"], st["up"], st["cache"], st["table"], st["lens"],
                                    st["max_new"], st["tokens"], st["scale"], workspace=space, device_error=st["err"])
    x = _rows(st)
    S, L, _ = x.shape
    T, H, _ = st["q"].shape
    n = st["max_new"]
    # every sequence's keys and values, and as many query rows as the one with most: [S, H, n, .]
    kv = torch.matmul(x[..., :LATENT].flatten(0, 1), st["up"].float().flatten(0, 1).T).view(S, L, H, NOPE + VALUE)
    k, v = kv[..., :NOPE].permute(0, 2, 3, 1), kv[..., NOPE:].transpose(1, 2)
    new = (st["cu"][1:] - st["cu"][:-1]).long()
    j = torch.arange(n, device=x.device)
    row = st["cu"][:-1].long()[:, None] + j
    q = st["q"][row.clamp(max=T - 1)].float().transpose(1, 2) * st["scale"]
    score = torch.matmul(q[..., :NOPE], k)
    score += torch.matmul(q[..., NOPE:], x[:, None, :, LATENT:].transpose(2, 3))
    seen = torch.arange(L, device=x.device) <= ((st["lens"].long() - new)[:, None] + j)[:, None, :, None]
    p, inv = _softmax_(score, seen)
    o = torch.matmul(p, v) * inv
    return o.transpose(1, 2)[st["seq"], st["place"]].to(st["q"].dtype)


def _heads(st, name, scale):
    """float32 [S, H, longest in whole blocks, D] of every sequence's rows."""
    return st[name].view(torch.uint8)[st["table"].long()].view(st[name].dtype).float().transpose(1, 2).flatten(2, 3) * scale


def _weights(st):
    if own:
        import paged_kv_cache_54_gb300 as pa
        S, Hq, D = st["q"].shape
        space = _workspace(st, lambda: pa.pa_decode_weights_workspace_size(S, Hq, st["case"]["kv_heads"], D,
                                                                           st["max_len"]))
        pa.pa_decode_weights(st["out"], st["new_weights"], st["q"], st["k"], st["v"], st["table"], st["lens"],
                             st["max_len"], st["scale"], weights_in=st["weights"], decay=0.75, k_scale=st["ks"],
                             v_scale=st["vs"], workspace=space, device_error=st["err"])
        return st["out"], st["new_weights"]
    S, Hq, D = st["q"].shape
    H, W = st["case"]["kv_heads"], st["max_len"]
    k = _heads(st, "k", st["ks"])[:, :, :W]
    seen = torch.arange(W, device=k.device) < st["lens"][:, None, None, None]
    score = torch.matmul(st["q"].float().view(S, H, -1, D) * st["scale"], k.transpose(2, 3))
    p, inv = _softmax_(score, seen)
    p *= inv
    v = torch.where(seen.transpose(2, 3), _heads(st, "v", st["vs"])[:, :, :W], 0.0)
    out = torch.matmul(p, v).view(S, Hq, D).to(st["q"].dtype)
    added = 0.75 * st["weights"] + p.sum(2)
    st["new_weights"].copy_(torch.where(seen[:, 0], added, st["new_weights"]))
    return out, st["new_weights"]


def _kept(weights, lens, budget, recent):
    """(kept tokens in order [S, H, budget], how many of each sequence): the
    last `recent`, then the largest weights, the lower index where they tie."""
    at = torch.arange(weights.shape[2], device=weights.device)
    n = lens.long()[:, None, None]
    key = torch.where(at >= n - recent, math.inf, weights)
    key = torch.where(at < n, key, -1.0)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    count = lens.clamp(max=budget)
    best = torch.where(torch.arange(best.shape[2], device=at.device) < count.long()[:, None, None], best,
                       weights.shape[2])
    best = torch.nn.functional.pad(best, (0, budget - best.shape[2]), value=weights.shape[2])
    return torch.sort(best, dim=-1).values, count


def _evict(st):
    case = st["case"]
    if own:
        import paged_kv_cache_54_gb300 as pa
        S, H, W = st["weights"].shape
        space = _workspace(st, lambda: pa.pa_evict_workspace_size(S, H, case["budget"]))
        pa.pa_evict_tokens(st["k"], st["v"], st["table"], st["lens"], st["weights"], st["new_table"], st["new_lens"],
                           st["new_weights"], case["budget"], case["recent"], workspace=space, device_error=st["err"])
        return st["k"], st["v"], st["new_lens"], st["new_weights"]
    bs = case["block"]
    kept, count = _kept(st["weights"], st["lens"], case["budget"], case["recent"])
    s, h, i = torch.nonzero(torch.arange(case["budget"], device="cuda") < count[:, None, None].expand(-1, kept.shape[1], 1),
                            as_tuple=True)
    j = kept[s, h, i]
    src, dst = st["table"][s, j // bs].long(), st["new_table"][s, i // bs].long()
    for c in (st["k"].view(torch.uint8), st["v"].view(torch.uint8)):
        c[dst, h, i % bs] = c[src, h, j % bs]
    st["new_weights"][s, h, i] = st["weights"][s, h, j]
    st["new_lens"].copy_(count)
    return st["k"], st["v"], st["new_lens"], st["new_weights"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op, bs = case["op"], case["block"]
    if op == "latent_write":
        out = st["cache"].double().view(-1, ROW)
        for t, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                out[slot] = torch.cat((st["latent"][t], st["rope"][t])).double()
        return out.view(st["cache"].shape)
    lens, table = st["lens"].tolist(), st["table"]
    if op == "latent_decode":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        n = case["new"]
        for s, L in enumerate(lens):
            x = st["cache"][table[s, : -(-L // bs)].long()].reshape(-1, ROW)[:L].double()
            for j in range(n):
                see = L - (n - 1 - j)
                if see > 0:
                    w = torch.softmax(st["q"][s, j].double() @ x[:see].T * st["scale"], -1)
                    out[s, j] = w @ x[:see, :LATENT]
        return out
    if op == "latent_prefill":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        cu = st["cu"].tolist()
        for s, L in enumerate(lens):
            x = st["cache"][table[s, : -(-L // bs)].long()].reshape(-1, ROW)[:L].double()
            q = st["q"][cu[s]:cu[s + 1]].double()
            hidden = torch.arange(L, device="cuda")[None] > (L - len(q) + torch.arange(len(q), device="cuda"))[:, None]
            for h in range(case["heads"]):
                kv = x[:, :LATENT] @ st["up"][h].double().T
                key = torch.cat((kv[:, :NOPE], x[:, LATENT:]), 1)
                w = torch.softmax((q[:, h] @ key.T * st["scale"]).masked_fill_(hidden, -math.inf), -1)
                out[cu[s]:cu[s + 1], h] = w @ kv[:, NOPE:]
        return out
    H, D = case["kv_heads"], case["head_dim"]

    def head(c, s, h, L):
        blocks = table[s, : -(-L // bs)].long()
        return c.view(torch.uint8)[blocks, h].view(c.dtype).reshape(-1, D)[:L].double()

    if op == "weights":
        G = case["q_heads"] // H
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        new = st["new_weights"].double()
        for s, L in enumerate(lens):
            for h in range(H if L else 0):
                q = st["q"][s, h * G:(h + 1) * G].double()
                w = torch.softmax(q @ (head(st["k"], s, h, L) * st["ks"]).T * st["scale"], -1)
                out[s, h * G:(h + 1) * G] = w @ (head(st["v"], s, h, L) * st["vs"])
                new[s, h, :L] = 0.75 * st["weights"][s, h, :L].double() + w.sum(0)
        return out, new
    k, v = st["k"].view(torch.uint8).clone(), st["v"].view(torch.uint8).clone()
    new = st["new_weights"].double()
    count = [min(L, case["budget"]) for L in lens]
    for s, L in enumerate(lens):
        w = st["weights"][s].cpu().numpy()[:, :L].astype(np.float64)
        w[:, max(0, L - case["recent"]):] = math.inf
        for h in range(H):
            order = np.lexsort((np.arange(L), -w[h]))[: count[s]]
            j = torch.from_numpy(np.sort(order)).cuda()
            i = torch.arange(count[s], device="cuda")
            src, dst = table[s][j // bs].long(), st["new_table"][s][i // bs].long()
            for c in (k, v):
                c[dst, h, i % bs] = c[src, h, j % bs]
            new[s, h, : count[s]] = st["weights"][s, h, j].double()
    k, v = k.view(st["k"].dtype), v.view(st["v"].dtype)
    wide = k.is_floating_point()
    return (k.double() if wide else k, v.double() if wide else v,
            torch.tensor(count, dtype=torch.int32, device="cuda"), new)
