"""GPU tests of the serving operators that send small inputs through every
kernel and every way of sharing out the work (tolerances as in
test_gpu_serving.py: the arithmetic is the same)."""
import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M

import _serving as ref
import test_gpu_serving as base

pytestmark = pytest.mark.gpu

DEV = "cuda"

# Rows of a KV head that the host announces: each picks another kernel
# (max_q picks the kernel only, whatever the lengths are).
ANNOUNCED = {"one tile of 8": 8, "tiles of 16": 32, "streams share keys": 512, "row pairs": 4096}


def _run(c, rows, **kw):
    c.max_q = max(1, rows // (c.heads // c.hkv))
    return c.run(**kw)


@pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)
@pytest.mark.parametrize("heads,hkv,d", [(8, 1, 128), (8, 8, 64), (10, 2, 64), (24, 2, 128)])
@pytest.mark.parametrize("lens", sorted(base.LENS))
def test_every_kernel_matches_64_bits(lens, heads, hkv, d, rows):
    c = base.Case(base.LENS[lens], heads, hkv, d, 32, seed=heads + d)
    for window in (0, 9):
        out, lse = _run(c, rows, window=window)
        base.check(c, out, lse, c.expect(d ** -0.5, window=window), window)


@pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)
@pytest.mark.parametrize("heads,hkv,d", [(8, 1, 128), (6, 2, 64)])
def test_every_kernel_on_prompts_behind_a_cached_prefix(heads, hkv, d, rows):
    c = base.Case([(700, 150), (129, 127), (0, 0), (1, 300)], heads, hkv, d, 64, seed=3)
    out, lse = _run(c, rows)
    base.check(c, out, lse, c.expect(d ** -0.5))
    again, lse2 = _run(c, rows)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)
def test_every_kernel_on_rows_that_see_nothing(rows):
    # more queries than cached tokens: the first ones stand before the row's start
    c = base.Case([(0, 20), (40, 3), (0, 9)], 8, 2, 64, 16, seed=5, seq=[7, 43, 0])
    out, lse = _run(c, rows)
    base.check(c, out, lse, c.expect(64 ** -0.5))
    assert not out[:13].any() and torch.isneginf(lse[:13]).all()


@pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_kernel_keeps_nan_to_queries_that_see_it(side, d, rows):
    c = base.Case([(50, 8), (30, 40), (170, 3)], 16, 2, d, 16, seed=6)
    for r, t in ((0, 54), (1, 33), (1, 66), (2, 120), (2, 171)):
        c.codes["kv".index(side), c.table[r, t // 16], :, t % 16, 5:9] = 0x7F
    out, lse = _run(c, rows)
    o, l, mag, span = c.expect(d ** -0.5)
    got = base._np(out.double())
    nan = np.isnan(l)[:, :, None] | np.zeros(o.shape, bool) if side == "k" else np.isnan(o)
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(base._np(lse)), np.isnan(l))
    assert np.array_equal(np.isnan(got), nan)
    lim = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -16 * span[:, :, None]) * mag
    assert (np.abs(got - o)[~nan] <= lim[~nan]).all()


@pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)
def test_every_kernel_on_extreme_scales(rows):
    for k_exp, v_exp, q_std, scale in (((-9, -6), (-50, 50), 1.0, 0.02),
                                       ((-50, -30), (-9, -6), 2.0 ** 30, 2.0 ** -4),
                                       ((20, 40), (-60, -58), 2.0 ** -40, 2.0 ** -3)):
        c = base.Case([(200, 1), (90, 6), (600, 2)], 16, 2, 128, 16, seed=8, k_exp=k_exp,
                      v_exp=v_exp, q_std=q_std)
        out, lse = _run(c, rows, scale=scale)
        base.check(c, out, lse, c.expect(scale), (k_exp, v_exp))


@pytest.mark.parametrize("heads,hkv,d", [(32, 32, 64), (64, 8, 128)])
def test_many_short_tiles_stay_whole(heads, hkv, d):
    # above 160 strips of 32 tokens a CTA, none of a tile's own above 40
    n = 128 if hkv == 32 else 400
    rng = np.random.default_rng(7)
    lens = [(int(x), 1) for x in rng.integers(180, 330, n)]
    c = base.Case(lens, heads, hkv, d, 32, seed=7)
    out, lse = c.run()
    base.check(c, out, lse, c.expect(d ** -0.5))


@pytest.mark.parametrize("tiles", [1, 3, 16])
@pytest.mark.parametrize("q", [1, 3])
def test_few_long_tiles_are_split_each_on_its_own(tiles, q):
    c = base.Case([(9001, q), (31, 1), (5000, q)], 8, 1, 64, 128, seed=tiles) if tiles < 16 else \
        base.Case([(2500, q)] * 8, 16, 2, 64, 64, seed=tiles)
    if tiles == 1:
        c = base.Case([(30000, q)], 4, 1, 64, 128, seed=1)
    out, lse = c.run()
    base.check(c, out, lse, c.expect(64 ** -0.5))
    again, _ = c.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("bs", [16, 64, 128])
def test_append_of_many_tokens(bs):
    """More than 1,024 tokens, so that a CTA's 64 slots hold few whole blocks or
    many; blocks that a thread block's registers do not hold; ragged ends."""
    d, hkv = 128, 2
    rng = np.random.default_rng(bs)
    lens = [(0, 3 * bs), (bs - 3, 400), (7, 1), (0, 1)] + [(5, 2)] * 40 + [(bs // 2, 700)]
    need = [-(-(c + n) // bs) for c, n in lens]
    n_blocks = sum(need) + 1
    ids = rng.permutation(n_blocks)
    slots, at = [], 0
    for (c, n), k in zip(lens, need):
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(c, c + n)]
        at += k
    slots[11:13] = [-1, -1]        # tokens that go nowhere, inside a block
    assert len(slots) > 1024
    codes = rng.integers(0, 127, (2, n_blocks, hkv, bs, d)).astype(np.uint8)
    scale = rng.integers(127 - 12, 127 - 3, (2, n_blocks, hkv)).astype(np.uint8)
    new = rng.standard_normal((2, len(slots), hkv, d)) * 2.0 ** rng.integers(
        -6, 4, (2, len(slots), 1, 1))
    t = [torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in new]
    k, v = torch.from_numpy(codes).to(DEV)
    ks, vs = torch.from_numpy(scale).to(DEV)
    # two calls, so that no two groups of one block are written at once
    cut = 13
    cache = M.KVCache(k, v, ks, vs)
    for lo, hi in ((0, cut), (cut, len(slots))):
        cache.append(t[0][lo:hi], t[1][lo:hi], base._dev(slots[lo:hi]))
        for s in range(2):
            codes[s], scale[s] = base.expect_append(codes[s], scale[s],
                                                    base._np(t[s][lo:hi].double()), slots[lo:hi], bs)
    for s, (c, sc) in enumerate(((k, ks), (v, vs))):
        assert np.array_equal(base._np(sc), scale[s]), s
        assert np.array_equal(base._np(c), codes[s]), s


@pytest.mark.parametrize("experts,k", [(256, 8), (896, 16), (1024, 32), (96, 12)])
@pytest.mark.parametrize("step", [0.0, 0.125])
def test_route_when_the_best_share_a_lane(experts, k, step):
    """The best experts are the ones that one lane holds (four in every 128, or
    one in every 32), descending or all equal: it looks again and again."""
    rng = np.random.default_rng(experts + k)
    x = rng.uniform(-6, -5, (16, experts))
    for r in range(16):
        lane = (5 * r) % 32
        mine = [e for e in range(experts) if (e % 128) // 4 == lane] if experts >= 128 else \
            [e for e in range(experts) if e % 32 == lane]
        for i, e in enumerate(mine):
            x[r, e] = 3.0 - step * i
    x = x.astype(np.float32)
    want_i, want_w = ref.route(x.astype(np.float64), None, k, "sigmoid", 1, 1, 1, True, 1.0)
    idx, w = M.moe_route(base._dev(x, torch.float32), k)
    assert np.array_equal(base._np(idx), want_i)
    np.testing.assert_allclose(base._np(w), want_w, rtol=1e-6)
