"""GPU tests of the serving operators against 64-bit restatements (_serving.py):
block tables and slot maps, the 8-bit cache's append and attention, routing.

Tolerances, fixed before the first run.  Attention: q is bf16/f16 and the
cache E4M3 times powers of two, so scores are exact products summed in fp32
(D 2^-24 of their absolute sum S, taken twice for the exponential's own
rounding); probabilities enter the second product in f16 (2^-11 each, taken
twice for sums of subnormal ones); the result is rounded once (2^-9 of itself
for bf16, 2^-12 for f16, taken twice).  Routing weights: fp32 arithmetic of
about ten roundings, 1e-6 relative."""
import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M

import _serving as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _np(t):
    return t.detach().cpu().numpy()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
class Case:
    """A random cache whose unused bytes are NaN codes, with tables over shuffled blocks."""

    def __init__(self, lens, heads, hkv, d, bs, dtype=torch.bfloat16, seed=0, k_exp=(-9, -6),
                 v_exp=(-9, -6), layout="head", spare=2, q_std=1.0, seq=None):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.hkv, self.d, self.bs, self.dtype = lens, heads, hkv, d, bs, dtype
        self.seq = np.array([c + n for c, n in lens] if seq is None else seq)
        need = [-(-int(s) // bs) for s in self.seq]
        self.mb = max(max(need), 1)
        self.n_blocks = sum(need) + spare
        ids = rng.permutation(self.n_blocks)
        self.table = np.full((len(lens), self.mb), -7, np.int64)
        codes = np.full((2, self.n_blocks, hkv, bs, d), 0x7F, np.uint8)
        scale = np.full((2, self.n_blocks, hkv), 255, np.uint8)
        at = 0
        for r, n in enumerate(need):
            for b in range(n):
                i = ids[at]
                at += 1
                self.table[r, b] = i
                used = min(bs, int(self.seq[r]) - b * bs)
                x = rng.standard_normal((2, hkv, used, d)) * 120.0
                codes[:, i, :, :used] = ref.e4m3_round(x)
                for s, (lo, hi) in enumerate((k_exp, v_exp)):
                    scale[s, i] = rng.integers(lo, hi + 1, hkv) + 127
        self.codes, self.scale = codes, scale
        self.q_start = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        q = rng.standard_normal((int(self.q_start[-1]), heads, d)) * q_std
        self.q = torch.from_numpy(q).to(dtype).to(DEV)
        self.layout = layout
        self.max_q = max(n for _, n in lens)

    def cache(self):
        k, v = torch.from_numpy(self.codes).to(DEV)
        if self.layout == "token":     # token-major blocks behind a head-major view
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif self.layout == "joint":   # K and V of a block side by side in one tensor
            kv = torch.stack([k, v], dim=1)
            k, v = kv[:, 0], kv[:, 1]
        ks, vs = torch.from_numpy(self.scale).to(DEV)
        return M.KVCache(k, v, ks, vs)

    def expect(self, scale, causal=True, window=0):
        q = _np(self.q.double())
        with np.errstate(invalid="ignore"):
            return ref.attention(q, ref.read_cache(self.codes[0], self.scale[0]),
                                 ref.read_cache(self.codes[1], self.scale[1]), self.table,
                                 self.seq, self.q_start, scale, causal, window, self.n_blocks)

    def run(self, cache=None, q=None, **kw):
        cache = cache or self.cache()
        return cache.attention(self.q if q is None else q, _dev(self.table), _dev(self.seq),
                               _dev(self.q_start), self.max_q, return_lse=True, **kw)


def check(c, out, lse, want, what=""):
    o, l, mag, span = want
    got = _np(out.double())
    u = 2.0 ** -8 if c.dtype == torch.bfloat16 else 2.0 ** -11
    rel = 2.0 ** -10 + 2 * c.d * 2.0 ** -24 * span[:, :, None]
    tol = u * np.abs(o) + rel * mag + 1e-30
    if c.dtype == torch.float16:
        tol = tol + 2.0 ** -24       # f16 subnormals
    assert np.array_equal(np.isnan(got), np.isnan(o)), what
    bad = np.abs(got - o) > tol
    assert not bad.any(), (what, np.argwhere(bad)[:5], got[bad][:5], o[bad][:5], tol[bad][:5])
    gl = _np(lse).astype(np.float64)
    assert np.array_equal(np.isneginf(gl), np.isneginf(l)), what
    fin = np.isfinite(l)
    err = np.abs(gl[fin] - l[fin])
    lim = 2.0 ** -20 + 2.0 ** -22 * np.abs(l[fin]) + c.d * 2.0 ** -24 * span[fin]
    assert (err <= lim).all(), (what, err.max())


HEADS = [(8, 1, 128), (8, 8, 64), (4, 2, 128), (7, 1, 64), (10, 2, 64), (32, 2, 128), (40, 1, 128)]
LENS = {
    "one": [(0, 1)],
    "decode": [(0, 1), (15, 1), (16, 1), (62, 1), (63, 1), (64, 1), (330, 1), (127, 1)],
    "verify": [(100, 8), (0, 3), (37, 5), (255, 1), (190, 8)],
    "prompt": [(0, 70), (33, 41)],
    "mixed": [(500, 1), (0, 37), (0, 0), (77, 2), (129, 17)],
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("heads,hkv,d", HEADS)
@pytest.mark.parametrize("lens", sorted(LENS))
def test_attention_matches_64_bits(lens, heads, hkv, d, dtype):
    c = Case(LENS[lens], heads, hkv, d, 16 if d == 64 else 64, dtype, seed=heads)
    out, lse = c.run()
    check(c, out, lse, c.expect(d ** -0.5))


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["head", "token", "joint"])
def test_attention_block_sizes_and_layouts(bs, layout):
    c = Case([(300, 1), (5, 2), (bs - 1, 1), (bs, 1), (2 * bs, 20)], 8, 2, 128, bs, seed=bs,
             layout=layout)
    out, lse = c.run()
    check(c, out, lse, c.expect(128 ** -0.5))


@pytest.mark.parametrize("window", [1, 2, 17, 64, 200, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows16", [True, False])
def test_attention_windows_and_full_masks(window, causal, rows16):
    heads = 4 if rows16 else 32
    c = Case([(300, 1), (40, 4), (0, 9), (513, 3), (130, 80)], heads, 2, 64, 32, seed=window)
    out, lse = c.run(causal=causal, window=window, scale=0.2)
    check(c, out, lse, c.expect(0.2, causal, window))


def test_attention_without_causal_mask():
    c = Case([(60, 5), (0, 40), (200, 1)], 8, 2, 128, 16, seed=3)
    out, lse = c.run(causal=False)
    check(c, out, lse, c.expect(128 ** -0.5, causal=False))


@pytest.mark.parametrize("heads", [4, 24])
def test_rows_that_see_nothing_give_zero(heads):
    """More queries than cached tokens (the first see nothing), and rows with none cached."""
    c = Case([(0, 5), (0, 30), (0, 2), (20, 3)], heads, 2, 128, 16, seed=4, seq=[2, 7, 0, 23])
    out, lse = c.run()
    want = c.expect(128 ** -0.5)
    assert np.isneginf(want[1][:3]).all()
    check(c, out, lse, want)
    out, lse = c.run(causal=False)
    check(c, out, lse, c.expect(128 ** -0.5, causal=False))


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("heads", [2, 24])
@pytest.mark.parametrize("window", [0, 9])
def test_nan_reaches_only_queries_that_see_it(side, heads, window):
    """NaN codes at some cached positions: queries before them (causal) or past them (window)
    stay exact, the others are NaN where the sum meets it."""
    c = Case([(50, 8), (30, 40), (170, 3)], heads, 2, 128, 16, seed=6)
    for r, t in ((0, 54), (1, 33), (1, 66), (2, 120), (2, 171)):
        c.codes["kv".index(side), c.table[r, t // 16], :, t % 16, 5:9] = 0x7F
    out, lse = c.run(window=window)
    o, l, mag, span = c.expect(128 ** -0.5, window=window)
    if side == "k":     # a NaN score makes the whole row NaN
        nan = np.isnan(l)
        assert nan.any() and not nan.all()
        assert np.array_equal(np.isnan(_np(lse)), nan)
        got = _np(out.double())
        assert np.isnan(got[nan]).all()
        keep = ~nan
        err = np.abs(got - o)[keep]
        lim = (2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -16 * span[:, :, None]) * mag)[keep]
        assert (err <= lim).all()
    else:
        assert np.isnan(o).any() and not np.isnan(o).all()
        got = _np(out.double())
        assert np.array_equal(np.isnan(got), np.isnan(o))
        keep = ~np.isnan(o)
        lim = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -16 * span[:, :, None]) * mag
        assert (np.abs(got - o)[keep] <= lim[keep]).all()


@pytest.mark.parametrize("heads", [4, 32])
def test_extreme_scales(heads):
    """Blocks whose V scales are 2^100 apart, with scores that favour the small ones, and
    tiny or huge keys and queries."""
    for k_exp, v_exp, q_std in (((-9, -6), (-50, 50), 1.0), ((-50, -30), (-9, -6), 2.0 ** 30),
                                ((20, 40), (-60, -58), 2.0 ** -40)):
        c = Case([(200, 1), (90, 6), (600, 2)], heads, 2, 128, 16, seed=8, k_exp=k_exp,
                 v_exp=v_exp, q_std=q_std)
        scale = 0.02 if k_exp[0] == -9 else 2.0 ** -4
        if k_exp[0] == 20:
            scale = 2.0 ** -3
        out, lse = c.run(scale=scale)
        check(c, out, lse, c.expect(scale), (k_exp, v_exp))


def test_block_ids_outside_the_cache_are_not_seen():
    c = Case([(100, 1), (100, 20)], 8, 2, 128, 16, seed=9)
    c.table[0, 2] = -1
    c.table[1, 1] = c.n_blocks
    c.table[1, 6] = 2 ** 31 - 1
    out, lse = c.run()
    check(c, out, lse, c.expect(128 ** -0.5))


@pytest.mark.parametrize("heads", [8, 48])
def test_long_rows_beside_short_ones(heads):
    """A row long enough to be split over many CTAs, beside short ones."""
    c = Case([(3, 1), (20011, 1), (100, 1), (4500, 2)], heads, 2, 128, 64, seed=10)
    out, lse = c.run()
    check(c, out, lse, c.expect(128 ** -0.5))


def test_strided_queries_and_outputs_another_stream_and_graph():
    c = Case([(300, 1), (40, 3), (70, 1)], 8, 2, 128, 32, seed=11)
    want = c.expect(128 ** -0.5)
    tokens = c.q.shape[0]
    fused = torch.zeros(tokens, 12, 128, dtype=c.dtype, device=DEV)   # q, k, v side by side
    fused[:, :8] = c.q
    out = torch.full((tokens, 10, 128), 7.0, dtype=c.dtype, device=DEV)
    cache, table, seq, qs = c.cache(), _dev(c.table), _dev(c.seq), _dev(c.q_start)
    wide = torch.full((3, c.mb + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :c.mb] = table
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, lse = cache.attention(fused[:, :8], wide[:, :c.mb], seq, qs, 3, out=out[:, 1:9],
                             return_lse=True, stream=st)
    st.synchronize()
    check(c, o, lse, want)
    assert (out[:, 0] == 7).all() and (out[:, 9] == 7).all()
    # captured once, replayed after the lengths changed on the device
    g = torch.cuda.CUDAGraph()
    static = torch.empty_like(c.q)
    with torch.cuda.graph(g):
        cache.attention(c.q, table, seq, qs, 3, out=static)
    static.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(c, static, lse, want)
    c.seq = c.seq - np.array([100, 0, 30])
    seq.copy_(_dev(c.seq))
    g.replay()
    o2, lse2 = c.run(cache=cache)
    torch.cuda.synchronize()
    check(c, static, lse2, c.expect(128 ** -0.5))


def test_attention_is_deterministic_and_ignores_padding_tokens():
    c = Case([(3000, 2), (900, 1)], 16, 2, 128, 64, seed=12)
    a = c.run()
    b = c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pad = torch.cat([c.q, c.q[:2]])
    out = torch.full_like(pad, 3.0)
    c.cache().attention(pad, _dev(c.table), _dev(c.seq), _dev(c.q_start), 2, out=out)
    assert torch.equal(out[:3], a[0]) and (out[3:] == 3).all()


def test_cache_offsets_past_32_bits():
    """Blocks more than 4 GiB apart in one tensor."""
    c = Case([(90, 1), (33, 20)], 8, 2, 128, 32, seed=13)
    step = 300 * 2 ** 20 // c.n_blocks * 16
    big = torch.zeros(step * (c.n_blocks - 1) + 4 * 2 * 32 * 128, dtype=torch.uint8, device=DEV)
    assert big.numel() > 2 ** 32
    inner = 2 * 32 * 128
    k, v = (torch.as_strided(big, (c.n_blocks, 2, 32, 128), (step, 32 * 128, 128, 1), o)
            for o in (0, inner))
    k.copy_(torch.from_numpy(c.codes[0]))
    v.copy_(torch.from_numpy(c.codes[1]))
    ks, vs = torch.from_numpy(c.scale).to(DEV)
    cache = M.KVCache(k, v, ks, vs)
    out, lse = c.run(cache=cache)
    check(c, out, lse, c.expect(128 ** -0.5))
    new = torch.randn(1, 2, 128, device=DEV).to(torch.bfloat16)
    last = c.n_blocks - 1
    cache.append(new, new, _dev([last * 32]))
    want = ref.e4m3_round(_np(new[0].double()) * 2.0 ** -np.array(
        [[ref.block_exp(float(x))] for x in new[0].abs().amax(dim=1)]))
    assert np.array_equal(_np(k[last, :, 0]), want) and np.array_equal(_np(v[last, :, 0]), want)


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
def expect_append(codes, scale, new, slots, bs):
    """codes [n_blocks, heads, bs, d], scale [n_blocks, heads]: updated copies."""
    codes, scale = codes.copy(), scale.copy()
    n_blocks, hkv = scale.shape
    t = 0
    while t < len(slots):
        b = slots[t] // bs
        e = t
        while e < len(slots) and slots[e] >= 0 and slots[e] // bs == b:
            e += 1
        if slots[t] < 0 or b >= n_blocks:
            t = max(e, t + 1)
            continue
        off = slots[t] % bs
        for h in range(hkv):
            x = new[t:e, h]
            fin = np.abs(x[np.isfinite(x)])
            ex = ref.block_exp(fin.max() if fin.size else 0.0)
            if off:
                old = int(np.clip(int(scale[b, h]) - 127, -60, 60))
                if old >= ex:
                    ex = old
                else:
                    codes[b, h, :off] = ref.e4m3_round(
                        ref.e4m3_table()[codes[b, h, :off]] * 2.0 ** (old - ex))
            scale[b, h] = ex + 127
            codes[b, h, off:off + e - t] = ref.e4m3_round(x * 2.0 ** -ex)
        t = e
    return codes, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("d,hkv,bs", [(128, 2, 64), (64, 3, 16), (128, 1, 128), (64, 8, 32)])
def test_append_matches_64_bits(d, hkv, bs, dtype):
    rng = np.random.default_rng(d + bs)
    lens = [(0, 1), (bs - 1, 3), (bs // 2, 1), (5, 4 * bs), (bs, 2), (3, 1), (0, 2 * bs + 1)]
    need = [-(-(c + n) // bs) for c, n in lens]
    n_blocks = sum(need) + 1
    ids = rng.permutation(n_blocks)
    slots, at = [], 0
    for (c, n), k in zip(lens, need):
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(c, c + n)]
        at += k
    slots += [-1, -1]
    codes = rng.integers(0, 256, (2, n_blocks, hkv, bs, d)).astype(np.uint8)
    codes[(codes & 127) == 127] = 3
    codes[0, 0, 0, 0, 0] = 0x7F                     # a NaN already stored stays one
    scale = rng.integers(127 - 12, 127 - 3, (2, n_blocks, hkv)).astype(np.uint8)
    new = rng.standard_normal((2, len(slots), hkv, d)) * 2.0 ** rng.integers(-6, 4, (2, len(slots), 1, 1))
    new[0, 1, 0, :4] = [0.0, -0.0, 1e-7, -3e-6]
    t = [torch.from_numpy(x).to(dtype).to(DEV) for x in new]
    k, v = torch.from_numpy(codes).to(DEV)
    ks, vs = torch.from_numpy(scale).to(DEV)
    M.KVCache(k, v, ks, vs).append(t[0], t[1], _dev(slots))
    for s, (c, sc) in enumerate(((k, ks), (v, vs))):
        wc, ws = expect_append(codes[s], scale[s], _np(t[s].double()), slots, bs)
        assert np.array_equal(_np(sc), ws), s
        assert np.array_equal(_np(c), wc), s


def test_append_special_values():
    """Zeros, subnormals, infinities and NaN, values past the scale range, exact powers of two."""
    bs, d = 16, 64
    rows = [np.zeros(d), np.full(d, 1e-40), np.full(d, 448.0), np.full(d, 449.0 * 4),
            np.full(d, 2.0 ** 100), np.full(d, 2.0 ** -100), np.full(d, 3.0)]
    rows[6][:5] = [np.inf, -np.inf, np.nan, -2.0, 0.5]
    rows.append(np.concatenate([np.arange(1, 33) / 16.0, -np.arange(1, 33) * 14.0]))
    x = torch.from_numpy(np.stack(rows)[:, None]).to(torch.bfloat16).to(DEV)
    n = len(rows)
    codes = np.full((n, 1, bs, d), 0x55, np.uint8)
    scale = np.full((n, 1), 255, np.uint8)
    slots = [i * bs for i in range(n)]
    k, v = (torch.from_numpy(codes).to(DEV) for _ in range(2))
    ks, vs = (torch.from_numpy(scale).to(DEV) for _ in range(2))
    M.KVCache(k, v, ks, vs).append(x, x, _dev(slots))
    wc, ws = expect_append(codes, scale, _np(x.double()), slots, bs)
    for c, s in ((k, ks), (v, vs)):
        got = _np(c)
        nan = (wc & 127) == 127
        assert np.array_equal((got & 127) == 127, nan)
        assert np.array_equal(got[~nan], wc[~nan]) and np.array_equal(_np(s), ws)


def test_append_strided_layouts_and_padded_slots():
    rng = np.random.default_rng(2)
    n, hkv, bs, d = 40, 2, 16, 128
    fused = torch.from_numpy(rng.standard_normal((n, 8, d))).to(torch.bfloat16).to(DEV)
    new_k, new_v = fused[:, 4:6], fused[:, 6:8]
    slots = np.concatenate([np.arange(7, 7 + n), np.full(24, -1)])
    base = [torch.zeros(6, bs, hkv, d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    k, v = (t.transpose(1, 2) for t in base)
    ks, vs = (torch.full((6, hkv), 100, dtype=torch.uint8, device=DEV) for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    M.KVCache(k, v, ks, vs).append(new_k, new_v, _dev(slots), stream=st)
    st.synchronize()
    for c, s, x in ((k, ks, new_k), (v, vs, new_v)):
        wc, ws = expect_append(np.zeros((6, hkv, bs, d), np.uint8), np.full((6, hkv), 100, np.uint8),
                               _np(x.double()), list(slots[:n]), bs)
        assert np.array_equal(_np(c), wc) and np.array_equal(_np(s), ws)


def test_append_skips_slots_outside_the_cache():
    x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((2, 1), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    M.KVCache(k, v, ks, vs).append(x, x, _dev([-1, 32, 2 ** 31 - 1, 16]))
    assert (k[0] == 0).all() and (k[1, 0, 1:] == 0).all() and (k[1, 0, 0] != 0).all()
    assert _np(ks).tolist() == [[127], [119]]


# ---------------------------------------------------------------------------
# Block tables
# ---------------------------------------------------------------------------
def _plan_case(ctx, q, bs, mb, n_free, n_slots, seed=0):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(100000).astype(np.int64)
    rows = len(ctx)
    table = np.full((rows, mb), -5, np.int64)
    at = n_free
    for r, c in enumerate(ctx):
        h = min(mb, -(-max(int(c), 0) // bs))
        table[r, :h] = ids[at:at + h]
        at += h
    free = ids[:max(n_free, 1)]
    want = ref.plan(ctx, q, table, free, n_free, bs, n_slots)
    t = _dev(table)
    p = M.kv_plan(_dev(ctx), _dev(q), t, _dev(free), _dev([n_free]), bs, n_slots)
    got = (_np(p.seq_lens), _np(p.q_start), _np(p.slot_map), int(p.n_free), int(p.n_unserved),
           _np(t))
    for g, w, name in zip(got, want, ("seq_lens", "q_start", "slot_map", "n_free", "n_unserved",
                                      "table")):
        assert np.array_equal(g, w), (name, g, w)


@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("rows", [1, 7, 513, 3000, 16384])
def test_plan_matches_row_by_row(bs, rows):
    rng = np.random.default_rng(rows)
    mb = 9
    ctx = rng.integers(0, bs * 7, rows)
    ctx[rng.random(rows) < 0.3] = rng.integers(0, 4) * bs    # full blocks
    q = np.where(rng.random(rows) < 0.7, 1, rng.integers(0, 2 * bs, rows))
    total = int(q.sum())
    need = int((-(-(ctx + q) // bs) - -(-ctx // bs)).sum())
    n_free = min(need + 3, 30000)
    _plan_case(ctx, q, bs, mb, n_free, total + 5, rows)


def test_plan_when_blocks_slots_or_table_run_out():
    ctx, q = [0, 60, 64, 10, 100, 0, 3], [40, 10, 1, 2, 30, 0, 1]
    for n_free in range(0, 8):
        _plan_case(ctx, q, 16, 9, n_free, 90)
    for n_slots in (0, 1, 39, 40, 41, 53, 83, 84):
        _plan_case(ctx, q, 16, 9, 20, n_slots)
    for mb in (1, 4, 5, 7, 8):
        c = [min(x, 16 * mb) for x in ctx]
        _plan_case(c, q, 16, mb, 20, 90)


def test_plan_negative_and_huge_lengths():
    _plan_case([5, -3, 4, 16], [3, 2, -1, 2 ** 31 - 20], 16, 4, 6, 12)


def test_release_pushes_blocks_and_plan_takes_them_again():
    bs, mb = 16, 4
    seq = [33, 5, 0, 64, 16]
    table = np.arange(20).reshape(5, 4) + 100
    fin = np.array([1, 0, 1, 1, 0], bool)
    free = np.concatenate([[7, 8, 9], np.full(12, -1)])
    t_seq, t_free, t_n = _dev(seq), _dev(free), _dev([3])
    M.kv_release(torch.from_numpy(fin).to(DEV), t_seq, _dev(table), t_free, t_n, bs)
    assert _np(t_seq).tolist() == [0, 5, 0, 0, 16]
    want = [7, 8, 9, 100, 101, 102, 112, 113, 114, 115]
    assert _np(t_free)[:10].tolist() == want and int(t_n) == 10
    t = _dev(table)
    p = M.kv_plan(t_seq, _dev([17, 1, 0, 0, 1]), t, t_free, t_n, bs, 32)
    assert _np(t)[0, :2].tolist() == [115, 114] and _np(t)[4, 1] == 113 and int(p.n_free) == 7
    # pushes past the end of the list are dropped
    short = _dev([1, 2])
    n = _dev([1])
    M.kv_release(torch.ones(5, dtype=torch.bool, device=DEV), _dev(seq), _dev(table), short, n, bs)
    assert _np(short).tolist() == [1, 100] and int(n) == 2


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------
ROUTES = [
    (64, 4, 1, 1, 1), (896, 16, 1, 1, 1), (256, 8, 8, 4, 2), (160, 6, 8, 3, 1), (60, 4, 1, 1, 2),
    (1024, 32, 1, 1, 1), (1, 1, 1, 1, 1), (33, 5, 3, 2, 2), (128, 8, 32, 7, 2), (512, 1, 16, 1, 2),
    (32, 32, 1, 1, 1), (32, 8, 32, 8, 2),
]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("experts,k,groups,topk_groups,group_top", ROUTES)
def test_route_matches_64_bits(experts, k, groups, topk_groups, group_top, with_bias, scoring):
    """Logits on a coarse grid: experts differ by far more than rounding or are exact ties."""
    rng = np.random.default_rng(experts + k)
    rows = 37
    x = rng.permuted(np.tile(np.linspace(-4, 4, experts), (rows, 1)), axis=1).astype(np.float32)
    x[1, :] = 0.5                                  # a row of ties
    if experts >= 4:
        x[2, ::3] = x[2, 0]
    # a bias that keeps sums on distinct values: a few experts lifted clear of the rest
    bias = np.where(np.arange(experts) % 11 == 3, 1.25, 0.0).astype(np.float32) if with_bias else None
    want_i, want_w = ref.route(x.astype(np.float64), bias, k, scoring, groups, topk_groups,
                               group_top, True, 2.5)
    for renorm in (True, False):
        idx, w = M.moe_route(_dev(x, torch.float32), k, bias=None if bias is None else
                             _dev(bias, torch.float32), scoring=scoring, n_groups=groups,
                             topk_groups=topk_groups, group_top=group_top, renormalize=renorm,
                             routed_scale=2.5)
        if not renorm:
            want_i, want_w = ref.route(x.astype(np.float64), bias, k, scoring, groups,
                                       topk_groups, group_top, False, 2.5)
        assert np.array_equal(_np(idx), want_i)
        np.testing.assert_allclose(_np(w), want_w, rtol=1e-6, atol=1e-12)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_route_types_strides_and_many_rows(dtype):
    rng = np.random.default_rng(5)
    rows, experts, k = 5003, 200, 6
    x = torch.from_numpy(rng.permuted(np.tile(np.arange(experts + 8) / 32.0 - 3, (rows, 1)),
                                      axis=1)).to(dtype).to(DEV)[:, 3:3 + experts]
    assert x.stride(0) == experts + 8
    idx, w = M.moe_route(x, k, scoring="softmax", renormalize=False)
    want_i, want_w = ref.route(_np(x.double()), None, k, "softmax", 1, 1, 1, False, 1.0)
    assert np.array_equal(_np(idx), want_i)
    np.testing.assert_allclose(_np(w), want_w, rtol=1e-6, atol=1e-12)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_masked_and_non_finite_logits(scoring):
    inf, nan, low = np.inf, np.nan, float(np.finfo(np.float32).min)
    x = np.array([[-inf] * 8, [low] * 8, [-inf, 1, -inf, 2, -inf, -inf, 0.5, -inf],
                  [low, 1, low, 2, low, low, low, low], [1, 2, 3, 4, 5, 6, 7, 8]], np.float32)
    want_i, want_w = ref.route(x.astype(np.float64), None, 3, scoring, 1, 1, 1, True, 1.0)
    idx, w = M.moe_route(_dev(x, torch.float32), 3, scoring=scoring)
    assert np.array_equal(_np(idx), want_i)
    np.testing.assert_allclose(_np(w), want_w, rtol=1e-6, atol=1e-12)
    if scoring == "sigmoid":        # a NaN comes last
        y = x[4:].copy()
        y[0, 7] = nan
        idx, w = M.moe_route(_dev(y, torch.float32), 8, scoring=scoring, renormalize=False)
        assert _np(idx)[0].tolist() == [6, 5, 4, 3, 2, 1, 0, 7] and np.isnan(_np(w)[0, 7])


def test_route_agrees_with_the_layers_router():
    """The layer's own selection (sigmoid, bias, top-k, renormalised to 2.5) from its logits."""
    from gen.configs import CONFIGS
    from moe_decode_step_gb300 import synthetic
    cfg = CONFIGS["tiny_b1"]
    weights = synthetic.make_weights(cfg)
    layer = synthetic.make_layer(cfg, max_batch=64, weights=weights)
    x, _ = synthetic.make_activations(cfg, B=32)
    idx, w = layer.router_topk(x)
    logits = x.float() @ weights["router_w"].float().T
    i2, w2 = M.moe_route(logits, cfg.top_k, bias=weights["router_bias"], routed_scale=2.5)
    same = (idx == i2).all(dim=1)
    assert same.sum() >= 31        # logits summed in another order may swap one near-tie
    torch.testing.assert_close(w[same], w2[same], rtol=1e-5, atol=1e-6)
    layer.close()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
def test_refusals_name_the_argument():
    c = Case([(40, 1)], 4, 2, 128, 16)
    cache, table, seq, qs = c.cache(), _dev(c.table), _dev(c.seq), _dev(c.q_start)
    good = dict(q=c.q, block_table=table, seq_lens=seq, q_start=qs, max_q=1)

    def refuses(match, exc=ValueError, **kw):
        with pytest.raises(exc, match=match):
            cache.attention(**{**good, **kw})
    refuses("q:", q=c.q.float())
    refuses("q:", q=c.q[..., :64])
    refuses("q:", q=c.q.cpu())
    refuses("seq_lens", seq_lens=seq.long())
    refuses("q_start", q_start=qs[:1])
    refuses("block_table", block_table=table[:, ::2])
    refuses("out", out=torch.empty_like(c.q)[:, :3])
    refuses("invalid", exc=M.MoEError, q=c.q[:, :3])            # 3 heads over 2 KV heads
    refuses("invalid", exc=M.MoEError, window=-1)
    odd = torch.zeros(1, 4 * 128 + 4, dtype=c.dtype, device=DEV)[:, 4:].view(1, 4, 128)
    refuses("unsupported", exc=M.MoEError, q=odd)               # 8-byte aligned queries
    k, v = torch.from_numpy(c.codes).to(DEV)
    ks, vs = torch.from_numpy(c.scale).to(DEV)
    with pytest.raises(ValueError, match="v:"):
        M.KVCache(k, v[:1], ks, vs)
    with pytest.raises(ValueError, match="k_scale"):
        M.KVCache(k, v, ks[:, :1], vs)
    with pytest.raises(ValueError, match="k:"):
        M.KVCache(k.float(), v, ks, vs)
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="slot_map"):
        cache.append(x, x, _dev([0]))
    with pytest.raises(ValueError, match="v:"):
        cache.append(x, x[:1], _dev([0, 1]))
    with pytest.raises(ValueError, match="k, v"):
        cache.append(x, x.half(), _dev([0, 1]))
    with pytest.raises(M.MoEError, match="unsupported"):
        cache.append(torch.zeros(2, 2, 132, dtype=torch.bfloat16, device=DEV)[..., 2:130], x,
                     _dev([0, 1]))
    with pytest.raises(M.MoEError, match="invalid"):
        M.kv_plan(seq, seq, table, seq, seq, 24, 4)
    with pytest.raises(ValueError, match="q_lens"):
        M.kv_plan(seq, qs, table, seq, seq, 16, 4)
    logits = torch.zeros(2, 64, device=DEV)
    for kw in (dict(top_k=65), dict(top_k=5, n_groups=16), dict(top_k=4, n_groups=7),
               dict(top_k=2, n_groups=4, topk_groups=5), dict(top_k=2, group_top=3)):
        with pytest.raises(M.MoEError, match="invalid"):
            M.moe_route(logits, **kw)
    with pytest.raises(M.MoEError, match="unsupported"):
        M.moe_route(torch.zeros(2, 1056, device=DEV), 4)
    with pytest.raises(ValueError, match="scoring"):
        M.moe_route(logits, 2, scoring="relu")
    with pytest.raises(ValueError, match="bias"):
        M.moe_route(logits, 2, bias=torch.zeros(63, device=DEV))


def test_empty_calls_do_nothing():
    c = Case([(40, 1)], 4, 2, 128, 16)
    cache = c.cache()
    q = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    out = cache.attention(q, _dev(c.table), _dev(c.seq), _dev([0, 0]), 0)
    assert out.shape == q.shape
    x = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    cache.append(x, x, _dev([]))
    idx, w = M.moe_route(torch.empty(0, 64, device=DEV), 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
