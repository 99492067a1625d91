"""Measured cases of the serving operators around the MoE decode layer: block tables and slot maps
(kv_plan), the 8-bit KV cache's append and attention (KVCache.append, KVCache.attention) and expert
routing from logits (moe_route).

`run` computes an operator in plain torch operations in 32 bits, or, where `own` is true, through
the package's entry points; `exact` restates the definitions in 64 bits.

The cache holds E4M3 codes with one E8M0 scale per (block of tokens, KV head); codes and scales come
back as torch's float8 types, which read as the numbers they stand for.
"""
import math

import torch

own = False

EXP_MIN, EXP_MAX = -60, 60      # scale exponents a cache block may take


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _attn(name, rows, q_lo, q_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, block, window=0,
          dtype="bfloat16"):
    return {"name": name, "op": "attention", "rows": rows, "q_lo": q_lo, "q_hi": q_hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "window": window, "dtype": dtype}


def _append(name, rows, q_lo, q_hi, ctx_lo, ctx_hi, kv_heads, dim, block, dtype="bfloat16"):
    return {"name": name, "op": "append", "rows": rows, "q_lo": q_lo, "q_hi": q_hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "kv_heads": kv_heads, "dim": dim, "block": block,
            "dtype": dtype}


def _plan(name, rows, q_lo, q_hi, prompts, ctx_lo, ctx_hi, block, max_blocks):
    return {"name": name, "op": "plan", "rows": rows, "q_lo": q_lo, "q_hi": q_hi,
            "prompts": prompts, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "block": block,
            "max_blocks": max_blocks}


def _route(name, rows, experts, top_k, scoring, bias, groups, topk_groups, group_top, renorm,
           dtype="float32"):
    return {"name": name, "op": "route", "rows": rows, "experts": experts, "top_k": top_k,
            "scoring": scoring, "bias": bias, "groups": groups, "topk_groups": topk_groups,
            "group_top": group_top, "renorm": renorm, "dtype": dtype}


def listed():
    return [
        # one user, a short context: the latency of a decode step's attention
        _attn("attn one row", 1, 1, 1, 332, 332, 64, 8, 128, 64),
        # a full decode batch of 64 rows over ragged contexts
        _attn("attn decode batch", 64, 1, 1, 2047, 16383, 64, 8, 128, 64),
        # a verify step: 8 sequences of an anchor token and 7 drafts
        _attn("attn verify", 8, 8, 8, 4090, 8185, 64, 8, 128, 64),
        # one user deep in a very long context, few KV heads: the split over the context
        _attn("attn long context", 1, 1, 1, 262142, 262142, 32, 2, 128, 64),
        # sliding-window layers with one KV head per query head
        _attn("attn window", 32, 1, 1, 500, 8000, 32, 32, 64, 16, window=1024, dtype="float16"),
        # prompts in chunks behind a cached prefix: the tensor-core regime
        _attn("attn prompt", 2, 2049, 4096, 4097, 8191, 32, 8, 128, 64),
        # every row of a decode batch writes one token into its partly filled block
        _append("append decode batch", 64, 1, 1, 100, 9000, 8, 128, 64),
        # prompts written into the cache
        _append("append prompts", 16, 517, 1531, 0, 300, 8, 128, 64),
        # block bookkeeping of a small decode batch and of a large mixed one
        _plan("plan decode", 8, 1, 1, 0, 40, 8000, 64, 256),
        _plan("plan mixed", 2048, 1, 511, 256, 0, 15000, 64, 256),
        # routing of a decode batch's rows (this layer's 16 of 896), and of a long prompt's tokens
        # with grouped selection (8 of 256 in 4 of 8 groups)
        _route("route decode", 64, 896, 16, "sigmoid", True, 1, 1, 1, True),
        _route("route prompt", 32768, 256, 8, "sigmoid", True, 8, 4, 2, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(64, 8, 128), (32, 8, 128), (32, 2, 128), (32, 32, 64), (16, 1, 128), (28, 4, 128),
          (40, 8, 64), (12, 12, 64), (8, 8, 128), (24, 8, 64)]


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "plan", "route"])
    if op == "attention":
        heads, kv_heads, dim = rng.choice(_HEADS)
        block = rng.choice([16, 32, 64, 128])
        window = rng.choice([0, 0, 0, _log_int(rng, 17, 4096)])
        dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
        kind = rng.choice(["decode", "verify", "prompt"])
        while True:
            if kind == "prompt":
                rows, q_hi = _log_int(rng, 1, 4), _log_int(rng, 65, 4096)
                ctx_hi = _log_int(rng, 1, 8191)
            else:
                rows = _log_int(rng, 1, 64)
                q_hi = 1 if kind == "decode" else rng.randint(2, 8)
                ctx_hi = _log_int(rng, 16, 262142 if rows == 1 else 16383)
            q_lo = q_hi if kind == "decode" else rng.randint(1, q_hi)
            ctx_lo = rng.randint(0, ctx_hi)
            c = _attn("", rows, q_lo, q_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, block, window,
                      dtype)
            w = work(c)
            if (w["bytes"] <= 1.2e9 and w["flops"] <= 5e11
                    and rows * heads * q_hi * (ctx_hi + q_hi) <= 3.2e9
                    and rows * kv_heads * dim * (ctx_hi + q_hi) <= 1.1e9):
                break
    elif op == "append":
        kv_heads, dim = rng.choice([(8, 128), (2, 128), (32, 64), (1, 128), (4, 64)])
        if rng.random() < 0.5:
            rows, q_hi = _log_int(rng, 1, 512), rng.randint(1, 8)
        else:
            rows, q_hi = _log_int(rng, 1, 16), _log_int(rng, 33, 1531)
        ctx_hi = _log_int(rng, 1, 9000)
        c = _append("", rows, rng.randint(1, q_hi), q_hi, rng.randint(0, ctx_hi), ctx_hi,
                    kv_heads, dim, rng.choice([16, 32, 64, 128]),
                    rng.choice(["bfloat16", "float16"]))
    elif op == "plan":
        rows = _log_int(rng, 1, 2048)
        block, max_blocks = rng.choice([(16, 1024), (32, 512), (64, 256), (128, 130)])
        ctx_hi = _log_int(rng, 10, 15000)
        q_hi = rng.choice([1, 8, _log_int(rng, 16, 511)])
        c = _plan("", rows, 1, q_hi, rng.randint(0, max(1, rows // 8)), rng.randint(0, ctx_hi),
                  ctx_hi, block, max_blocks)
    else:
        experts, groups = rng.choice([(896, 1), (256, 8), (64, 1), (160, 8), (128, 4), (60, 1),
                                      (384, 1), (512, 16)])
        topk_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, topk_groups * (experts // groups)))
        scoring = rng.choice(["sigmoid", "softmax"])
        rows = _log_int(rng, 1, 32768 if experts <= 256 else 8192)
        c = _route("", rows, experts, top_k, scoring, rng.random() < 0.6, groups, topk_groups,
                   rng.choice([1, 2]), rng.random() < 0.7,
                   rng.choice(["float32", "float32", "bfloat16"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# Lengths (from the case alone, so that work() knows them; prepare() orders them by the seed)
# ---------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(c):
    """[(ctx, q)] per row."""
    n = c["rows"]
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], n)
    if c["op"] == "plan":   # `prompts` rows of up to q_hi new tokens, the others one token each
        q = [1] * n
        for i, v in enumerate(_spread(c["q_lo"], c["q_hi"], c["prompts"]) if c["prompts"] else []):
            q[(i * 7) % n if n > 7 else i % n] = v
        return list(zip(ctx, q))
    q = _spread(c["q_lo"], c["q_hi"], n)
    return list(zip(ctx, q[::2] + q[1::2]))


def work(case):
    c = case
    if c["op"] == "route":
        size = 2 if c["dtype"] == "bfloat16" else 4
        t, e = c["rows"], c["experts"]
        return {"bytes": t * e * size + (4 * e if c["bias"] else 0) + t * c["top_k"] * 8,
                "flops": 4 * t * e}
    lens = _lens(c)
    total = sum(q for _, q in lens)
    if c["op"] == "plan":
        bs = c["block"]
        need = sum(-(-(a + q) // bs) - -(-a // bs) for a, q in lens)
        held = sum(1 for a, q in lens if a % bs)     # a partly filled block's table entry
        return {"bytes": 16 * len(lens) + 8 * need + 4 * held + 4 * _slots(total), "flops": 0}
    hkv, d, bs = c["kv_heads"], c["dim"], c["block"]
    if c["op"] == "append":
        # codes and scales written; the codes a block already holds are read only where its scale
        # grows, which the inputs decide, so they are not counted
        blocks = sum(-(-(a + q) // bs) - a // bs for a, q in lens)
        return {"bytes": total * hkv * d * (2 * 2 + 2) + 2 * blocks * hkv + 4 * total, "flops": 0}
    win, heads = c["window"], c["heads"]
    seen = pairs = 0
    for a, q in lens:
        seen += min(a + q, q - 1 + win) if win else a + q   # tokens at least one query sees
        if not win:
            pairs += q * a + q * (q + 1) // 2
        else:
            grow = max(0, min(q, win - 1 - a))              # queries that see their whole prefix
            pairs += grow * a + grow * (grow + 1) // 2 + (q - grow) * win
    return {"bytes": seen * hkv * 2 * d + 2 * seen // bs * hkv + total * heads * (4 * d + 4),
            "flops": 4 * d * heads * pairs}


def _slots(total):
    """Entries of a slot map: a step's buffers are sized in steps of 256 tokens."""
    return (total + 255) // 256 * 256


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within the cache's range."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _codes(v, e):
    """E4M3 codes (as float8) of v / 2^e; e broadcasts."""
    return torch.ldexp(v, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e8m0(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _bytes(t):
    return t.view(torch.uint8)


def _random_side(g, n_blocks, hkv, bs, d, spread):
    v = torch.randn(n_blocks, hkv, bs, d, generator=g, device="cuda")
    v *= torch.exp(spread * torch.randn(n_blocks, hkv, 1, 1, generator=g, device="cuda"))
    v *= torch.exp(0.4 * torch.randn(1, hkv, 1, d, generator=g, device="cuda"))   # channels differ
    e = _exponent(v.abs().amax(dim=(2, 3)))
    return _codes(v, e[:, :, None, None]), _e8m0(e)


def _tables(g, lens, bs, order, spare):
    """Block tables of the rows' whole lengths over shuffled block ids, int32 [rows, widest]."""
    need = [-(-(a + q) // bs) for a, q in lens]
    n_blocks = sum(need) + spare
    ids = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(max(need), 1), dtype=torch.int32, device="cuda")
    at = 0
    for r in range(len(lens)):
        k = need[order[r]]
        table[r, :k] = ids[at:at + k]
        at += k
    return table, n_blocks


def _cache(s, k, ks, v, vs):
    s.update(k=k, k_scale=ks, v=v, v_scale=vs)
    if own:   # the program's cache object over the same tensors
        import moe_decode_step_gb300 as M
        s["cache"] = M.KVCache(k, v, ks, vs)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        t, e = c["rows"], c["experts"]
        dt = getattr(torch, c["dtype"])
        bias = (0.05 * torch.randn(e, generator=g, device="cuda")) if c["bias"] else None
        logits = (1.3 * torch.randn(t, e, generator=g, device="cuda")).to(dt)
        for _ in range(12):   # rows where rounding could decide the selection are drawn again
            bad = _near_tie(c, logits, bias)
            logits = torch.where(bad[:, None], (1.3 * torch.randn(
                t, e, generator=g, device="cuda")).to(dt), logits)
        bad = _near_tie(c, logits, bias)
        ramp = torch.linspace(-3, 3, e, device="cuda", dtype=torch.float64)
        if bias is not None:   # evenly spaced biased scores, for a row that never came out clear
            want = torch.linspace(0.3, 0.7, e, device="cuda", dtype=torch.float64) - bias.double()
            ramp = torch.logit(want) if c["scoring"] == "sigmoid" else ramp
        s.update(logits=torch.where(bad[:, None], ramp.to(dt)[None], logits), bias=bias)
        return s
    lens = _lens(c)
    order = torch.randperm(len(lens), generator=torch.Generator().manual_seed(seed)).tolist()
    ctx, q = [lens[i][0] for i in order], [lens[i][1] for i in order]
    total, bs = sum(q), c["block"]
    s.update(ctx_lens=_ints(ctx), q_lens=_ints(q))
    if c["op"] == "plan":
        mb = c["max_blocks"]
        have = [-(-a // bs) for a in ctx]
        need = sum(-(-(a + n) // bs) - h for a, n, h in zip(ctx, q, have))
        spare = 64 + len(lens)
        ids = torch.randperm(sum(have) + need + spare, generator=g, device="cuda").to(torch.int32)
        held = torch.arange(mb, device="cuda")[None] < _ints(have)[:, None]
        table = torch.full((len(lens), mb), -1, dtype=torch.int32, device="cuda")
        table[held] = ids[:sum(have)]
        s.update(block_table=table, free_list=ids[sum(have):].clone(),
                 n_free=_ints([need + spare]), n_slots=_slots(total))
        return s
    hkv, d = c["kv_heads"], c["dim"]
    dt = getattr(torch, c["dtype"])
    if c["op"] == "append":
        # only the blocks this step touches are in the cache: a row's table begins at the block
        # its context ends in
        near = [(a % bs, n) for a, n in lens]
        table, n_blocks = _tables(g, near, bs, order, 3)
        pos = torch.cat([torch.arange(a % bs, a % bs + n) for a, n in zip(ctx, q)]).cuda()
        row = torch.repeat_interleave(torch.arange(len(q)), torch.tensor(q)).cuda()
        slots = table[row, pos // bs].long() * bs + pos % bs
        k, ks = _random_side(g, n_blocks, hkv, bs, d, 0.3)
        v, vs = _random_side(g, n_blocks, hkv, bs, d, 0.3)
        s.update(slot_map=slots.to(torch.int32),
                 new_k=(1.5 * torch.randn(total, hkv, d, generator=g, device="cuda")).to(dt),
                 new_v=torch.randn(total, hkv, d, generator=g, device="cuda").to(dt))
        _cache(s, k, ks, v, vs)
        return s
    table, n_blocks = _tables(g, lens, bs, order, 3)
    k, ks = _random_side(g, n_blocks, hkv, bs, d, 0.1)
    v, vs = _random_side(g, n_blocks, hkv, bs, d, 0.5)
    start = [0]
    for n in q:
        start.append(start[-1] + n)
    s.update(q=torch.randn(total, c["heads"], d, generator=g, device="cuda").to(dt),
             block_table=table, seq_lens=_ints([a + n for a, n in zip(ctx, q)]),
             q_start=_ints(start), max_q=max(q), scale=1.0 / math.sqrt(d))
    _cache(s, k, ks, v, vs)
    return s


def _near_tie(c, logits, bias):
    """Rows in which two scores that the selection compares are closer than rounding, but not
    equal by having equal inputs."""
    x = logits.double()
    p = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, dim=1)
    sel = p if bias is None else p + bias.double()
    t, e = sel.shape
    near = torch.zeros(t, dtype=torch.bool, device=sel.device)

    def close(v, n):   # among the n + 1 largest
        v = v.sort(dim=1, descending=True).values[:, :n + 1]
        gap = v[:, :-1] - v[:, 1:]
        size = v[:, 1:].abs() + (0.0 if bias is None else bias.abs().max().double())
        return ((gap > 0 if bias is None else gap >= 0) & (gap < 4e-6 * size)).any(dim=1)

    if c["groups"] > 1:
        per = sel.view(t, c["groups"], -1)
        score = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        near |= close(score, c["topk_groups"])
        keep = _best(score, c["topk_groups"])
        mask = torch.zeros(t, c["groups"], dtype=torch.bool, device=sel.device)
        mask.scatter_(1, keep, True)
        sel = sel.masked_fill(~mask.repeat_interleave(e // c["groups"], dim=1), -math.inf)
    return near | close(sel, min(c["top_k"], e - 1))


def _best(v, n):
    """Indices of each row's n largest, largest first, ties to the lower index."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import moe_decode_step_gb300 as M
        if op == "route":
            return M.moe_route(s["logits"], c["top_k"], bias=s["bias"], scoring=c["scoring"],
                               n_groups=c["groups"], topk_groups=c["topk_groups"],
                               group_top=c["group_top"], renormalize=c["renorm"],
                               routed_scale=2.5)
        if op == "plan":
            p = M.kv_plan(s["ctx_lens"], s["q_lens"], s["block_table"], s["free_list"],
                          s["n_free"], c["block"], s["n_slots"])
            return [s["block_table"], p.seq_lens, p.q_start, p.slot_map, p.n_free, p.n_unserved]
        if op == "append":
            s["cache"].append(s["new_k"], s["new_v"], s["slot_map"])
            return [s["k"], s["k_scale"], s["v"], s["v_scale"]]
        return s["cache"].attention(s["q"], s["block_table"], s["seq_lens"], s["q_start"],
                                    s["max_q"], scale=s["scale"], window=c["window"],
                                    return_lse=True)
    return {"route": _plain_route, "plan": _plain_plan, "append": _plain_append,
            "attention": _plain_attention}[op](s, c)


def _plain_route(s, c):
    x = s["logits"].float()
    t, e = x.shape
    if c["scoring"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        p = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
    sel = p if s["bias"] is None else p + s["bias"]
    if c["groups"] > 1:
        per = sel.view(t, c["groups"], -1)
        score = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]].sum(dim=2)
        mask = torch.zeros(t, c["groups"], dtype=torch.bool, device=x.device)
        mask.scatter_(1, _best(score, c["topk_groups"]), True)
        sel = sel.masked_fill(~mask.repeat_interleave(e // c["groups"], dim=1), -math.inf)
    idx = _best(sel, c["top_k"])
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return [idx.to(torch.int32), 2.5 * w]


def _plain_plan(s, c):
    ctx, q, bs = s["ctx_lens"].long(), s["q_lens"].long(), c["block"]
    table, n_free = s["block_table"], s["n_free"].long()
    mb = table.shape[1]
    have = (ctx + bs - 1) // bs
    total = (ctx + q + bs - 1) // bs
    fits = total <= mb
    need = (total - have) * fits
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= n_free))
    start = upto - need
    col = torch.arange(mb, device=table.device)[None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None]) & served[:, None]
    at = (n_free - 1 - (start[:, None] + col - have[:, None])).clamp(0, s["free_list"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_list"][at], table))
    seq = torch.where(served, ctx + q, ctx)
    q_end = torch.cumsum(q, 0)
    q_start = torch.cat([torch.zeros_like(q_end[:1]), q_end])
    i = torch.arange(s["n_slots"], device=table.device)
    row = torch.searchsorted(q_end, i, right=True).clamp_max(ctx.numel() - 1)
    pos = ctx[row] + i - q_start[row]
    slot = table[row, (pos // bs).clamp(0, mb - 1)] * bs + pos % bs
    slot = torch.where((i < q_end[-1]) & served[row], slot, torch.full_like(slot, -1))
    used = (need * served).sum()
    return [table, seq.to(torch.int32), q_start.to(torch.int32), slot.to(torch.int32),
            (n_free - used).to(torch.int32), (~served).sum().to(torch.int32).view(1)]


def _plain_append(s, c):
    bs = c["block"]
    slot = s["slot_map"].long()
    block, off = slot // bs, slot % bs
    out = []
    n_blocks, hkv = s["k"].shape[:2]
    # tokens a block holds before this step; blocks this step does not touch keep all of theirs
    first = torch.full((n_blocks,), bs, device=slot.device).scatter_reduce(
        0, block, off, "amin", include_self=True)
    touched = first < bs
    held = torch.arange(bs, device=slot.device)[None] < first[:, None]
    for codes, scale, new in ((s["k"], s["k_scale"], s["new_k"]),
                              (s["v"], s["v_scale"], s["new_v"])):
        x = new.float()
        amax = torch.zeros(n_blocks, hkv, device=x.device).scatter_reduce(
            0, block[:, None].expand(-1, hkv), x.abs().amax(dim=2), "amax", include_self=True)
        old = _bytes(scale).int() - 127
        e = _exponent(amax)
        e = torch.where((first > 0)[:, None], torch.maximum(old, e), e)
        e = torch.where(touched[:, None], e, old)
        shifted = _codes(codes.float(), (e - old)[:, :, None, None])
        _bytes(codes).copy_(torch.where(held[:, None, :, None], _bytes(shifted), _bytes(codes)))
        _bytes(codes)[block, :, off] = _bytes(_codes(x, e[block][:, :, None]))
        _bytes(scale).copy_((e + 127).to(torch.uint8))
        out += [codes, scale]
    return out


def _gathered(codes, scale, table):
    """[rows, kv_heads, tokens, dim] of the tables' blocks."""
    t = table.long()
    e = _bytes(scale).int()[t] - 127
    v = torch.ldexp(_bytes(codes)[t].view(torch.float8_e4m3fn).float(), e[..., None, None])
    r, n, h, bs, d = v.shape
    return v.permute(0, 2, 1, 3, 4).reshape(r, h, n * bs, d)


def _plain_attention(s, c):
    table, seq, q_start = s["block_table"], s["seq_lens"].long(), s["q_start"].long()
    hkv, d = c["kv_heads"], c["dim"]
    total, heads = s["q"].shape[:2]
    rows, mq = seq.numel(), s["max_q"]
    q_len = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=seq.device)
    at = (q_start[:-1, None] + i[None]).clamp_max(total - 1)
    q = s["q"][at].float().view(rows, mq, hkv, heads // hkv, d).permute(0, 2, 3, 1, 4)
    k = _gathered(s["k"], s["k_scale"], table)
    n = k.shape[2]
    x = torch.matmul(q.reshape(rows, hkv, -1, d), k.transpose(2, 3)).mul_(s["scale"])
    del k
    x = x.view(rows, hkv, heads // hkv, mq, n)
    pos = (seq - q_len)[:, None] + i[None]
    j = torch.arange(n, device=seq.device)
    seen = j[None, None] <= pos[:, :, None]
    if c["window"]:
        seen &= j[None, None] > pos[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(dim=4, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    x = x.sub_(m).exp_()
    z = x.sum(dim=4, keepdim=True)
    v = _gathered(s["v"], s["v_scale"], table)
    held = j[None] < seq[:, None]
    v = v * held[:, None, :, None]
    o = torch.matmul(x.view(rows, hkv, -1, n), v).view(rows, hkv, heads // hkv, mq, d)
    o = o / torch.where(z > 0, z, torch.ones_like(z))
    lse = (m + torch.log(z)).squeeze(4)
    t = torch.arange(total, device=seq.device)
    row = torch.searchsorted(q_start[1:], t, right=True)
    o = o.permute(0, 3, 1, 2, 4)[row, t - q_start[row]].reshape(total, heads, d)
    lse = lse.permute(0, 3, 1, 2)[row, t - q_start[row]].reshape(total, heads)
    return [o.to(s["q"].dtype), lse]


# ---------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None       # whole numbers only
    s = prepare(c, seed)
    return {"route": _exact_route, "append": _exact_append, "attention": _exact_attention}[
        c["op"]](s, c)


def _exact_route(s, c):
    x = s["logits"].double().cpu()
    t, e = x.shape
    p = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, dim=1)
    key = p.clone() if s["bias"] is None else p + s["bias"].double().cpu()
    if c["groups"] > 1:
        size = e // c["groups"]
        parts = key.reshape(t, c["groups"], size)
        score = parts.topk(min(c["group_top"], size), dim=2).values.sum(dim=2)
        order = torch.argsort(score, dim=1, descending=True, stable=True)
        for n in range(c["topk_groups"], c["groups"]):
            parts[torch.arange(t), order[:, n]] = -math.inf
        key = parts.reshape(t, e)
    idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :c["top_k"]]
    w = torch.take_along_dim(p, idx, 1)
    return [idx, 2.5 * (w / w.sum(dim=1, keepdim=True) if c["renorm"] else w)]


def _round_e4m3(x):
    """Nearest E4M3 value (ties to the even code, magnitudes past 448 to 448) of doubles."""
    a = x.abs().clamp_max(448.0)
    ex = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    ex = torch.where(torch.exp2(ex) > a, (ex - 1).clamp_min(-6), ex)
    step = torch.exp2(ex - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_append(s, c):
    bs, out = c["block"], []
    slots = s["slot_map"].long().cpu()
    block, off = slots // bs, slots % bs
    cut = [0] + [i for i in range(1, len(slots)) if block[i] != block[i - 1]] + [len(slots)]
    for codes, scale, new in ((s["k"], s["k_scale"], s["new_k"]),
                              (s["v"], s["v_scale"], s["new_v"])):
        val = codes.double().cpu()
        unit = torch.exp2(_bytes(scale).double().cpu() - 127)
        x = new.double().cpu()
        for a, b in zip(cut[:-1], cut[1:]):
            n, held = int(block[a]), int(off[a])
            want = torch.clamp(torch.ceil(torch.log2(x[a:b].abs().amax(dim=(0, 2)) / 448.0)),
                               EXP_MIN, EXP_MAX)
            u = torch.exp2(want)
            u = torch.maximum(u, unit[n]) if held else u
            val[n, :, :held] = _round_e4m3(val[n, :, :held] * (unit[n] / u)[:, None, None])
            val[n, :, held:held + b - a] = _round_e4m3(
                x[a:b].transpose(0, 1) / u[:, None, None])
            unit[n] = u
        out += [val, unit]
    return out


def _exact_attention(s, c):
    bs, hkv, d, win = c["block"], c["kv_heads"], c["dim"], c["window"]
    heads = s["q"].shape[1]
    grp = heads // hkv
    start, seq = s["q_start"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    for r, n in enumerate(seq):
        a, b = start[r], start[r + 1]
        ids = s["block_table"][r, :(n + bs - 1) // bs].long()
        pos = torch.arange(n - (b - a), n, device="cuda")
        j = torch.arange(n, device="cuda")
        hide = j[None] > pos[:, None]
        if win:
            hide |= j[None] <= pos[:, None] - win
        for h in range(hkv):
            def side(codes, scale):
                v = _bytes(codes)[ids, h].view(torch.float8_e4m3fn).double()
                u = torch.exp2(_bytes(scale)[ids, h].double() - 127)
                return (v * u[:, None, None]).reshape(-1, d)[:n]
            k, v = side(s["k"], s["k_scale"]), side(s["v"], s["v_scale"])
            for i in range(h * grp, (h + 1) * grp):
                x = s["q"][a:b, i].double() @ k.T * s["scale"]
                x[hide] = -math.inf
                lse[a:b, i] = torch.logsumexp(x, dim=1)
                out[a:b, i] = torch.exp(x - lse[a:b, i, None]) @ v
    return [out, lse]
