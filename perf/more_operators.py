"""Measured cases of the 8-bit operators around the MoE layer for prompts and decode steps: the
norm with the residual's addition and 8-bit outputs (rms_norm, fp8_quantize), matrix products in
8 bits (fp8_linear), tokens sorted by their experts (moe_dispatch), the products of experts with
ragged numbers of rows (expert_linear) and the weighted sum of their results (moe_combine).

`run` computes an operator in plain torch operations in 32 bits, or, where `own` is true, through
the package's entry points; `exact` restates the definitions in 64 bits.

8-bit activations and weights are E4M3 codes with E8M0 scales: one scale per (row, 128 columns) of
activations, one per (128 rows, 128 columns) of weights.  MXFP4 weights are the layer's canonical
layout: E2M1 nibbles, the lower column in the lower nibble, one E8M0 scale per (row, 32 columns).
Codes and scales come back as torch's float8 types, which read as the numbers they stand for.
"""
import math

import torch

own = False

EXP_MIN, EXP_MAX = -126, 120    # exponents of an activation's or an 8-bit weight's scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _norm(name, rows, d, residual=True, norm=True, out=True, codes=True, dtype="bfloat16"):
    return {"name": name, "op": "norm", "rows": rows, "d": d, "residual": residual, "norm": norm,
            "out": out, "codes": codes, "dtype": dtype}


def _linear(name, rows, n, k, swiglu=False, quantize=False, weights="e4m3", dtype="bfloat16"):
    """n: output columns (with swiglu the weights have 2 n rows: gates, then ups)."""
    return {"name": name, "op": "linear", "rows": rows, "n": n, "k": k, "swiglu": swiglu,
            "quantize": quantize, "weights": weights, "dtype": dtype}


def _experts(name, tokens, top_k, experts, n, k, gather, swiglu, quantize, weights,
             dtype="bfloat16"):
    return {"name": name, "op": "experts", "tokens": tokens, "top_k": top_k, "experts": experts,
            "n": n, "k": k, "gather": gather, "swiglu": swiglu, "quantize": quantize,
            "weights": weights, "dtype": dtype}


def _dispatch(name, tokens, top_k, experts):
    return {"name": name, "op": "dispatch", "tokens": tokens, "top_k": top_k, "experts": experts}


def _combine(name, tokens, top_k, experts, d, residual=True, dtype="bfloat16"):
    return {"name": name, "op": "combine", "tokens": tokens, "top_k": top_k, "experts": experts,
            "d": d, "residual": residual, "dtype": dtype}


def listed():
    return [
        # one user's token between attention and the experts: latency
        _norm("norm one row", 1, 7168),
        # a prompt's tokens: the router reads the 16-bit output, the experts the 8-bit one
        _norm("norm prompt", 8192, 7168),
        # the attention's output projection (64 heads of 128) of one token: weights streamed
        _linear("linear one row", 1, 7168, 8192),
        # queries, keys and values (64 + 2 * 8 heads of 128) of a full decode batch
        _linear("linear decode batch", 64, 10240, 7168),
        # the output projection of a long prompt
        _linear("linear prompt", 8192, 7168, 8192),
        # a verify step of 8 tokens through the MXFP4 experts: gates and ups, 8-bit results
        _experts("experts decode", 8, 16, 896, 2048, 7168, True, True, True, "mxfp4"),
        # a prompt through 8-bit experts: gates and ups, then (of MXFP4 experts) the way down
        _experts("experts prompt up", 4096, 8, 128, 2048, 4096, True, True, True, "e4m3"),
        _experts("experts prompt down", 4096, 8, 128, 7168, 2048, False, False, False, "mxfp4"),
        # a decode batch's and a long prompt's choices, sorted by expert
        _dispatch("dispatch decode", 64, 16, 896),
        _dispatch("dispatch prompt", 32768, 8, 256),
        # the experts' results of a decode batch and of a prompt, weighted, on the residual
        _combine("combine decode", 64, 16, 896, 7168),
        _combine("combine prompt", 4096, 8, 256, 7168),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_POOLS = [(64, 4), (896, 16), (256, 8), (128, 8), (60, 4), (16, 2), (8, 2), (160, 6)]


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "experts", "experts", "dispatch", "combine"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    while True:
        if op == "norm":
            norm = rng.random() < 0.8
            out, codes = rng.choice([(True, True), (False, True), (True, False)]) if norm else (
                False, True)
            c = _norm("", _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1024),
                      norm and rng.random() < 0.7, norm, out, codes, dtype)
        elif op == "linear":
            swiglu = rng.random() < 0.3
            weights = rng.choice(["e4m3", "e4m3", "mxfp4"])
            k = 128 * _log_int(rng, 2, 64) if weights == "mxfp4" else 16 * _log_int(rng, 8, 512)
            n = _log_int(rng, 65, 10240)
            c = _linear("", _log_int(rng, 1, 8192), n, k, swiglu, swiglu and rng.random() < 0.7,
                        weights, dtype)
        elif op == "experts":
            experts, top_k = rng.choice(_POOLS)
            swiglu = rng.random() < 0.5
            weights = rng.choice(["e4m3", "mxfp4"])
            c = _experts("", _log_int(rng, 1, 4096), top_k, experts, 128 * _log_int(rng, 2, 56),
                         128 * _log_int(rng, 2, 56), swiglu or rng.random() < 0.3, swiglu,
                         swiglu and rng.random() < 0.8, weights, dtype)
            rows, wide = c["tokens"] * top_k, c["n"] * c["k"] * (2 if swiglu else 1)
            if min(rows, experts) * wide > 4e9 or experts * wide > 2.6e10:
                continue
        else:
            experts, top_k = rng.choice(_POOLS)
            if op == "dispatch":
                c = _dispatch("", _log_int(rng, 1, 32768), top_k, experts)
            else:
                c = _combine("", _log_int(rng, 1, 8192), top_k, experts,
                             8 * _log_int(rng, 8, 1024), rng.random() < 0.6, dtype)
        w = work(c)
        if w["bytes"] <= 5.4e8 and w["flops"] <= 1.1e12:
            break
    del c["name"]
    return c


def _blocks(n):
    return (n + 127) // 128


def _routing(c):
    """The case's choices, int64 [tokens, top_k], distinct in a row; some experts are chosen more
    often than others.  From the case alone, so that work() knows how many experts are touched;
    prepare() orders tokens and experts by the seed."""
    t, k, e = c["tokens"], c["top_k"], c["experts"]
    g = torch.Generator().manual_seed(t * 1000003 + k * 1009 + e)
    score = torch.randn(1, e, generator=g) * 0.35 + torch.empty(t, e).exponential_(
        generator=g).log_().neg_()
    return torch.topk(score, k, dim=1).indices


def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        n, size = c["rows"] * c["d"], 2
        byts = n * size * (1 + 2 * c["residual"] + c["out"]) + c["norm"] * c["d"] * size
        if c["codes"]:
            byts += n + c["rows"] * _blocks(c["d"])
        return {"bytes": byts, "flops": 0}
    if op == "dispatch":
        n = c["tokens"] * c["top_k"]
        return {"bytes": 12 * n + 4 * (c["experts"] + 1), "flops": 0}
    if op == "combine":
        n = c["tokens"]
        return {"bytes": n * c["top_k"] * (2 * c["d"] + 8) + 2 * n * c["d"] * (1 + c["residual"]),
                "flops": 2 * n * c["top_k"] * c["d"]}
    k, n = c["k"], c["n"]
    wide = n * (2 if c["swiglu"] else 1)
    if op == "linear":
        rows = x_rows = c["rows"]
        touched, table = 1, 0
    else:
        rows = c["tokens"] * c["top_k"]
        x_rows = c["tokens"] if c["gather"] else rows
        touched = torch.unique(_routing(c)).numel()
        table = 4 * (c["experts"] + 1) + (4 * rows if c["gather"] else 0)
    weights = wide * k // 2 + wide * k // 32 if c["weights"] == "mxfp4" else (
        wide * k + _blocks(wide) * _blocks(k))
    out = rows * (n + _blocks(n)) if c["quantize"] else 2 * rows * n
    return {"bytes": touched * weights + x_rows * (k + _blocks(k)) + out + table,
            "flops": 2 * rows * wide * k}


# ---------------------------------------------------------------------------------------------
# 8-bit and 4-bit values
# ---------------------------------------------------------------------------------------------
def _bytes(t):
    return t.view(torch.uint8)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, within a scale's range."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _e8m0(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _quantize(v):
    """Codes and scales of fp32 [rows, d]: a scale per (row, 128 columns)."""
    rows, d = v.shape
    b = _blocks(d)
    p = v if d == 128 * b else torch.nn.functional.pad(v, (0, 128 * b - d))
    p = p.view(rows, b, 128)
    e = _exponent(p.abs().amax(dim=2))
    codes = torch.ldexp(p, -e[..., None]).clamp(-448.0, 448.0).view(rows, -1)[:, :d]
    return codes.to(torch.float8_e4m3fn), _e8m0(e)


def _rows(codes, scales, kind=torch.float32):
    """Values of activations: codes [rows, d], scales [rows, blocks]."""
    v = codes.to(kind)
    s = torch.exp2(_bytes(scales).to(kind) - 127).repeat_interleave(128, dim=-1)
    return v * s[..., :v.shape[-1]]


def _weights(w, s, kind=torch.float32):
    """Values of weights [..., n, k]: 8-bit with a scale per 128 x 128, or MXFP4."""
    unit = torch.exp2(_bytes(s).to(kind) - 127)
    if w.dtype == torch.uint8:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=kind, device=w.device)
        pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], dim=1)
        v = pairs[w.int()].flatten(-2)
        return v.unflatten(-1, (-1, 32)).mul_(unit[..., None]).flatten(-2)
    v = w.to(kind)
    n, k = v.shape[-2:]
    if n % 128 == 0 and k % 128 == 0:
        tiles = v.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
        return tiles.mul_(unit[..., :, None, :, None]).flatten(-2).flatten(-3, -2)
    unit = unit.repeat_interleave(128, dim=-2).repeat_interleave(128, dim=-1)
    return v * unit[..., :n, :k]


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _activations(g, rows, d):
    """Normal values whose channels and rows differ in size, a few channels standing out."""
    v = torch.randn(rows, d, generator=g, device="cuda")
    size = torch.exp(0.5 * torch.randn(1, d, generator=g, device="cuda"))
    size *= torch.where(torch.rand(1, d, generator=g, device="cuda") < 0.004, 12.0, 1.0)
    return v * size * torch.exp(0.2 * torch.randn(rows, 1, generator=g, device="cuda"))


def _make_weights(g, c, count):
    """Weights of `count` matrices [wide, k] (count 0: one, without that dimension)."""
    wide, k = c["n"] * (2 if c["swiglu"] else 1), c["k"]
    lead = (count,) if count else ()
    if c["weights"] == "mxfp4":
        # blocks of 32 normal values divided by their largest fill the eight magnitudes evenly
        w = torch.empty(lead + (wide, k // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty(lead + (wide, k // 32), dtype=torch.uint8, device="cuda")
        w.view(torch.int32).random_(-2 ** 31, 2 ** 31, generator=g)
        low = int(round(124.5 - 0.5 * math.log2(k)))
        s.random_(low - 1, low + 2, generator=g)
        return w, s.view(torch.float8_e8m0fnu)
    b, nb = _blocks(k), _blocks(wide)
    w = torch.empty(lead + (wide, k), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(lead + (nb, b), dtype=torch.float8_e8m0fnu, device="cuda")
    for i in range(max(count, 1)):
        v = torch.randn(128 * nb, 128 * b, generator=g, device="cuda").mul_(k ** -0.5)
        v[wide:] = 0
        v[:, k:] = 0
        v = v.view(nb, 128, b, 128)
        e = _exponent(v.abs().amax(dim=(1, 3)))
        codes = torch.ldexp(v, -e[:, None, :, None]).view(128 * nb, 128 * b)[:wide, :k]
        (w[i] if count else w).copy_(codes.to(torch.float8_e4m3fn))
        _bytes(s[i] if count else s).copy_(_bytes(_e8m0(e)))
    return w, s


def prepare(case, seed):
    c = case
    op = c["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    dt = getattr(torch, c.get("dtype", "bfloat16"))
    if op == "norm":
        s["x"] = _activations(g, c["rows"], c["d"]).to(dt)
        if c["norm"]:
            s["gamma"] = (1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
        s["residual"] = _activations(g, c["rows"], c["d"]).to(dt) if c["residual"] else None
        return s
    if op == "linear":
        s["x"], s["x_scales"] = _quantize(_activations(g, c["rows"], c["k"]))
        s["w"], s["w_scales"] = _make_weights(g, c, 0)
        return s
    t, k, e = c["tokens"], c["top_k"], c["experts"]
    names = torch.randperm(e, generator=g, device="cuda")
    idx = names[_routing(c).cuda()[torch.randperm(t, generator=g, device="cuda")]]
    if op == "dispatch":
        s["idx"] = idx.to(torch.int32)
        return s
    offsets, rows, slots = _plain_dispatch(idx, e)
    if op == "combine":
        s.update(y=torch.randn(t * k, c["d"], generator=g, device="cuda").to(dt), slots=slots)
        w = torch.rand(t, k, generator=g, device="cuda") + 0.1
        s["w"] = 2.5 * w / w.sum(dim=1, keepdim=True)
        s["residual"] = (torch.randn(t, c["d"], generator=g, device="cuda").to(dt)
                         if c["residual"] else None)
        return s
    s["x"], s["x_scales"] = _quantize(_activations(g, t if c["gather"] else t * k, c["k"]))
    s["w"], s["w_scales"] = _make_weights(g, c, e)
    most = torch.bincount(idx.flatten(), minlength=e).max().item()
    s.update(offsets=offsets, rows=rows if c["gather"] else None, most=most)
    return s


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import moe_decode_step_gb300 as M
        dt = getattr(torch, c.get("dtype", "bfloat16"))
        if op == "norm":
            if not c["norm"]:
                return list(M.fp8_quantize(s["x"]))
            r = M.rms_norm(s["x"], s["gamma"], residual=s["residual"], eps=1e-6, out=c["out"],
                           quantize=c["codes"])
            return [s["residual"], r.out, r.codes, r.scales]
        if op == "dispatch":
            return list(M.moe_dispatch(s["idx"], c["experts"]))
        if op == "combine":
            return M.moe_combine(s["y"], s["w"], s["slots"], residual=s["residual"])
        act = "swiglu" if c["swiglu"] else None
        if op == "linear":
            r = M.fp8_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], activation=act,
                             quantize=c["quantize"], out_dtype=dt)
        else:
            r = M.expert_linear(s["x"], s["x_scales"], s["w"], s["w_scales"], s["offsets"],
                                rows=s["rows"], activation=act, quantize=c["quantize"],
                                out_dtype=dt)
        return list(r) if c["quantize"] else r
    if op == "dispatch":
        return _plain_dispatch(s["idx"], c["experts"])
    return {"norm": _plain_norm, "linear": _plain_linear, "experts": _plain_experts,
            "combine": _plain_combine}[op](s, c)


def _plain_norm(s, c):
    z = s["x"].float()
    if not c["norm"]:
        return list(_quantize(z))
    if c["residual"]:
        z = z + s["residual"].float()
        s["residual"].copy_(z)
    y = z * torch.rsqrt(z.square().mean(dim=1, keepdim=True) + 1e-6) * s["gamma"].float()
    codes = _quantize(y) if c["codes"] else (None, None)
    return [s["residual"], y.to(s["x"].dtype) if c["out"] else None, *codes]


def _finish(y, c):
    """The product [rows, wide] as the operator returns it."""
    if c["swiglu"]:
        gate, up = y.chunk(2, dim=1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    if c["quantize"]:
        return list(_quantize(y))
    return y.to(getattr(torch, c["dtype"]))


def _plain_linear(s, c):
    x = _rows(s["x"], s["x_scales"])
    return _finish(torch.matmul(x, _weights(s["w"], s["w_scales"]).T), c)


def _plain_experts(s, c):
    rows = c["tokens"] * c["top_k"]
    i = torch.arange(rows, device="cuda")
    start = s["offsets"].long()
    expert = torch.searchsorted(start[1:], i, right=True)
    x = _rows(s["x"], s["x_scales"])
    if c["gather"]:
        x = x[s["rows"].long()]
    if rows <= c["experts"]:   # a matrix for each row
        w = _weights(s["w"][expert], _bytes(s["w_scales"])[expert])
        return _finish(torch.matmul(w, x[:, :, None]).squeeze(2), c)
    at = start[:-1, None] + torch.arange(s["most"], device="cuda")   # rows of each expert, padded
    x = x[at.clamp_max(rows - 1)]
    y = torch.matmul(x, _weights(s["w"], s["w_scales"]).transpose(1, 2))
    return _finish(y[expert, i - start[expert]], c)


def _plain_dispatch(idx, experts):
    flat = idx.flatten()
    by, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=by.device, dtype=by.dtype))
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(
        flat.numel(), device=by.device))
    return [offsets.to(torch.int32), (order // idx.shape[1]).to(torch.int32),
            slots.view(idx.shape).to(torch.int32)]


def _plain_combine(s, c):
    z = (s["y"].float()[s["slots"].long()] * s["w"][..., None]).sum(dim=1)
    if c["residual"]:
        z = z + s["residual"].float()
    return z.to(s["y"].dtype)


# ---------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "dispatch":
        return None       # whole numbers only
    s = prepare(c, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "experts": _exact_experts,
            "combine": _exact_combine}[c["op"]](s, c)


def _round_e4m3(x):
    """Nearest E4M3 value (ties to the even code, magnitudes past 448 to 448) of doubles."""
    a = x.abs().clamp_max(448.0)
    ex = torch.floor(torch.log2(a.clamp_min(2.0 ** -6)))
    ex = torch.where(torch.exp2(ex) > a, (ex - 1).clamp_min(-6), ex)
    step = torch.exp2(ex - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_quantize(y):
    codes = torch.empty_like(y)
    scales = []
    for j in range(0, y.shape[1], 128):
        part = y[:, j:j + 128]
        top = part.abs().amax(dim=1).clamp_min(1e-300)
        unit = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(EXP_MIN, EXP_MAX))
        codes[:, j:j + 128] = _round_e4m3(part / unit[:, None])
        scales.append(unit)
    return [codes, torch.stack(scales, dim=1)]


def _exact_norm(s, c):
    z = s["x"].double()
    if not c["norm"]:
        return _exact_quantize(z)
    if c["residual"]:
        z = z + s["residual"].double()
    y = z / torch.sqrt((z * z).sum(dim=1, keepdim=True) / c["d"] + 1e-6) * s["gamma"].double()
    codes = _exact_quantize(y) if c["codes"] else [None, None]
    return [z if c["residual"] else None, y if c["out"] else None, *codes]


def _exact_finish(y, c):
    if c["swiglu"]:
        gate, up = y[:, :c["n"]], y[:, c["n"]:]
        y = gate * torch.sigmoid(gate) * up
    return _exact_quantize(y) if c["quantize"] else y


def _exact_linear(s, c):
    x = _exact_rows(s["x"], s["x_scales"])
    y = [x @ _exact_matrix(s["w"], s["w_scales"], a, a + 1024).T
         for a in range(0, s["w"].shape[0], 1024)]
    return _exact_finish(torch.cat(y, dim=1), c)


def _exact_rows(codes, scales):
    v = codes.double()
    for j in range(scales.shape[1]):
        v[:, 128 * j:128 * j + 128] *= scales[:, j:j + 1].double()
    return v


def _exact_matrix(w, s, a, b):
    """Rows [a, b) of a weight matrix (a a multiple of 128)."""
    w = w[a:b]
    if w.dtype == torch.uint8:
        v = torch.zeros(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=w.device)
        for half, code in ((0, w & 15), (1, w >> 4)):
            mag = code & 7
            e = (mag >> 1).double()
            m = (mag & 1).double()
            size = torch.where(mag < 2, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
            v[:, half::2] = torch.where(code > 7, -size, size)
        for j in range(s.shape[1]):
            v[:, 32 * j:32 * j + 32] *= s[a:b, j:j + 1].double()
        return v
    v = w.double()
    for i in range(0, w.shape[0], 128):
        for j in range(s.shape[1]):
            v[i:i + 128, 128 * j:128 * j + 128] *= s[(a + i) // 128, j].double()
    return v


def _exact_experts(s, c):
    start = s["offsets"].tolist()
    x = _exact_rows(s["x"], s["x_scales"])
    if c["gather"]:
        x = x[s["rows"].long()]
    y = torch.zeros(x.shape[0], c["n"] * (2 if c["swiglu"] else 1), dtype=torch.float64,
                    device="cuda")
    for e in range(c["experts"]):
        a, b = start[e], start[e + 1]
        if a < b:
            y[a:b] = x[a:b] @ _exact_matrix(s["w"][e], s["w_scales"][e], 0, y.shape[1]).T
    return _exact_finish(y, c)


def _exact_combine(s, c):
    z = s["residual"].double() if c["residual"] else 0.0
    for j in range(c["top_k"]):
        z = z + s["w"][:, j:j + 1].double() * s["y"][s["slots"][:, j].long()].double()
    return z
