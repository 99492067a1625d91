"""GPU tests of the serving operators at the edges of what their calls accept:
block scales at both ends of their range, keys that lead the softmax by far,
scores so large that fp32 steps over whole octaves, lengths past 31 bits.
Attention goes through all four kernels; tolerances as in test_gpu_serving.py."""
import numpy as np
import pytest
import torch

import moe_decode_step_gb300 as M

import _serving as ref
import test_gpu_serving as base
from test_gpu_serving_paths import ANNOUNCED, _run

pytestmark = pytest.mark.gpu

DEV = "cuda"
every_kernel = pytest.mark.parametrize("rows", ANNOUNCED.values(), ids=ANNOUNCED)


# ---------------------------------------------------------------------------
# Attention: large scores
# ---------------------------------------------------------------------------
def _scores(c, r, i, h):
    """Scores (times scale 1) of query i of row r, head h, over the row's cached tokens, and
    the largest sum of magnitudes."""
    k = ref.read_cache(c.codes[0], c.scale[0])
    j = np.arange(int(c.seq[r]))
    kk = k[c.table[r, j // c.bs], h // (c.heads // c.hkv), j % c.bs]
    q = base._np(c.q.double())[c.q_start[r] + i, h]
    return kk @ q, (np.abs(kk) @ np.abs(q)).max()


@every_kernel
@pytest.mark.parametrize("v_exp", [(-9, -6), (-60, -40), (40, 60)])
@pytest.mark.parametrize("log_q", [18, 22, 25, 28, 34, 60])
def test_large_scores_take_the_best_key(log_q, v_exp, rows):
    """Scores of about 2^log_q, whose own fp32 spacing is up to 2^36: a softmax over them is
    the best key wherever it leads by more than the scores' rounding (d 2^-24 of their absolute
    sum) and 30 nats; the result is then its value, rounded once."""
    c = base.Case([(200, 1), (90, 6), (600, 2), (3, 40)], 16, 2, 128, 16, seed=log_q, v_exp=v_exp,
                  q_std=2.0 ** (log_q - 3.0))
    out, lse = _run(c, rows, scale=1.0, causal=False)
    got, gl = base._np(out.double()), base._np(lse).astype(np.float64)
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    v = ref.read_cache(c.codes[1], c.scale[1])
    seen = 0
    for r, (_, n) in enumerate(c.lens):
        for i in range(n):
            for h in range(c.heads):
                s, span = _scores(c, r, i, h)
                top = np.argsort(s)[::-1][:2]
                noise = 2 * c.d * 2.0 ** -24 * span
                t = c.q_start[r] + i
                assert abs(gl[t, h] - s[top[0]]) <= noise + np.log(len(s)) + 2.0 ** -22 * abs(s[top[0]])
                if s[top[0]] - s[top[1]] < 2 * noise + 30:
                    continue
                seen += 1
                j = top[0]
                want = v[c.table[r, j // c.bs], h // 8, j % c.bs]
                # beside the result's rounding the weight's own, and e^-30 of every other value
                rest = len(s) * np.exp(-30.0) * np.nanmax(np.abs(v[c.table[r, :-(-len(s) // c.bs)], h // 8]))
                assert (np.abs(got[t, h] - want) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(want) + rest).all()
    assert seen > 300


@every_kernel
def test_rows_beside_a_row_of_large_scores_stay_exact(rows):
    """One query and one head of huge values among ordinary ones of the same tile."""
    c = base.Case([(300, 1), (64, 7), (5, 30)], 16, 2, 128, 32, seed=2)
    q = c.q.clone()
    q[:, 3] *= 2.0 ** 30
    q[4] *= 2.0 ** 40
    plain = c.expect(128 ** -0.5)
    out, lse = _run(c, rows, q=q)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    keep = np.ones(plain[1].shape, bool)
    keep[:, 3] = keep[4] = False
    o, l, mag, span = (x[keep][:, None] for x in plain)
    base.check(c, out[torch.from_numpy(keep).to(DEV)][:, None], lse[torch.from_numpy(keep).to(DEV)][:, None],
               (o, l, mag, span))


# ---------------------------------------------------------------------------
# Attention: a key that leads
# ---------------------------------------------------------------------------
def _leading(lead, value_exp, heads=16, n=4096, q=1, d=128, seed=0):
    """A row whose first key leads the others by some `lead` nats; its values are zeros, or in a
    block whose scale is `value_exp` octaves above the others'."""
    c = base.Case([(n - q, q)], heads, 2, d, 16, seed=seed, k_exp=(-9, -9), v_exp=(-8, -8), q_std=0.25)
    c.q[:, :, 0] = 8.0
    k, v = c.codes
    k[:, :, :, 0] = np.where((k[:, :, :, 0] & 127) == 127, k[:, :, :, 0], 0)   # dim 0 is the lead's alone
    first = c.table[0, 0]
    k[first, :, 0] = 0
    k[first, :, 0, 0] = 0x7E                        # 448 * 2^-9 * 8 = 7
    if value_exp:
        c.scale[1, first] += value_exp
    else:
        v[first, :, 0] = 0
    return c, lead / 7.0


@every_kernel
@pytest.mark.parametrize("lead,value_exp", [(10, 0), (14, 0), (15, 0), (16, 0), (17, 0), (18, 0),
                                            (8, 6), (8, 10), (0, 14)])
def test_keys_behind_a_leading_one_keep_their_bits(lead, value_exp, rows):
    for q in (1, 5):
        c, scale = _leading(lead, value_exp, q=q, seed=lead + value_exp)
        out, lse = _run(c, rows, scale=scale)
        base.check(c, out, lse, c.expect(scale), (lead, value_exp, q))


# ---------------------------------------------------------------------------
# Attention: block scales at the ends of their range
# ---------------------------------------------------------------------------
@every_kernel
@pytest.mark.parametrize("behind", [0, 4, 8, 20, 40])
def test_small_values_count_in_the_denominator(behind, rows):
    """One key at V exponent 60, the others at -60 and `behind` bits behind it: their weights are
    2^-120 of its own beside the values, but count in full in the sum."""
    for heads, lo in ((16, -60), (2, -60), (16, -29), (16, -28)):
        c = base.Case([(1000, 1), (300, 3)], heads, 2, 128, 16, seed=1, k_exp=(-9, -9), v_exp=(lo, lo),
                      q_std=0.0)
        for r in range(2):
            first = c.table[r, 0]
            c.scale[1, first] = 60 + 127
            c.codes[0, first, :, 0] = 0
            c.codes[0, first, :, 0, 0] = 0x7E       # 448 * 2^-9
            c.codes[1, first, :, 1:] = 0            # the block's other values are zeros
        c.q[:, :, 0] = 8.0
        for b in range(c.n_blocks):
            c.codes[0, b, :, :, 0] = np.where((c.codes[0, b, :, :, 0] & 127) == 127,
                                              c.codes[0, b, :, :, 0], 0)
        for r in range(2):
            c.codes[0, c.table[r, 0], :, 0, 0] = 0x7E
        scale = max(behind, 1e-3) * np.log(2.0) / 7.0
        out, lse = _run(c, rows, scale=scale)
        base.check(c, out, lse, c.expect(scale), (heads, lo))


@every_kernel
def test_scales_over_the_whole_range(rows):
    for v_exp in ((-60, 60), (-60, -20), (-30, -26), (-60, -60)):
        c = base.Case([(200, 1), (90, 6), (600, 2)], 16, 2, 128, 16, seed=8, v_exp=v_exp)
        out, lse = _run(c, rows, scale=0.02)
        base.check(c, out, lse, c.expect(0.02), v_exp)


@every_kernel
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_query_that_sees_only_blocks_outside_the_cache_gives_zero(bad, rows):
    """... whatever the query holds; and one that sees some keys is as without the others."""
    c = base.Case([(31, 1), (100, 3), (20, 40)], 8, 2, 128, 32, seed=4)
    c.table[0] = -1
    c.table[1, :2] = c.n_blocks
    q = c.q.clone()
    q[0, 2] = bad
    q[0, 5, 7] = -bad
    out, lse = _run(c, rows, q=q)
    base.check(c, out, lse, c.expect(128 ** -0.5))
    assert not out[0].any() and torch.isneginf(lse[0]).all()


# ---------------------------------------------------------------------------
# Attention: what the host announces
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("max_q", [-2 ** 31, -1000, 0, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("window", [0, 9])
def test_any_announced_length_gives_the_same_result(max_q, window):
    c = base.Case([(100, 1)] * 64 + [(40, 3)], 16, 8, 64, 16, seed=5)
    c.max_q = max_q
    out, lse = c.run(window=window)
    base.check(c, out, lse, c.expect(64 ** -0.5, window=window))


# ---------------------------------------------------------------------------
# Block tables
# ---------------------------------------------------------------------------
PLAN_ROWS = """
import sys
sys.path[:0] = {path!r}
import numpy as np, test_gpu_serving as base
rows = {rows}
base._plan_case(np.full(rows, 5), np.ones(rows, int), 16, 2, 3, rows)
"""


@pytest.mark.parametrize("rows", [6109, 6110, 6143, 6144])
def test_plan_needs_no_larger_plan_before_it(rows):
    """Rows at which the kernel's shared memory passes 48 KB, each as a process's first plan."""
    import subprocess
    import sys
    p = subprocess.run([sys.executable, "-c", PLAN_ROWS.format(path=sys.path, rows=rows)],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


def test_plan_lengths_past_31_bits_are_not_served():
    """A table wide enough for them: the row keeps its length, its tokens go nowhere."""
    bs, mb = 128, 2 ** 24 + 8
    table = torch.zeros(2, mb, dtype=torch.int32, device=DEV)
    ctx = base._dev([2 ** 31 - 100, 5])
    p = M.kv_plan(ctx, base._dev([200, 1]), table, base._dev([3, 4]), base._dev([2]), bs, 300)
    assert base._np(p.seq_lens).tolist() == [2 ** 31 - 100, 6] and int(p.n_unserved) == 1
    slots = base._np(p.slot_map)
    assert (slots[:200] == -1).all() and slots[200] == 5 and (slots[201:] == -1).all()
    assert int(p.n_free) == 2


def test_plan_block_ids_whose_slots_pass_31_bits_map_nowhere():
    ids = [2 ** 27, 2 ** 27 + 1, -2 ** 28, 2 ** 31 - 1, -2 ** 31, 2 ** 27 - 1]
    p = M.kv_plan(base._dev([3] * 6), base._dev([1] * 6), base._dev(ids)[:, None], base._dev([0]),
                  base._dev([0]), 16, 6)
    slots = base._np(p.slot_map).astype(np.int64)
    assert (slots[:5] < 0).all() and slots[5] == (2 ** 27 - 1) * 16 + 3


def test_plan_fills_a_slot_map_of_any_length():
    n = 2 ** 31 - 1
    p = M.kv_plan(base._dev([3]), base._dev([2]), base._dev([[7]]), base._dev([0]), base._dev([0]), 16, n)
    assert base._np(p.slot_map[:3]).tolist() == [115, 116, -1]
    tail = p.slot_map[2:]
    assert all(int(x.max()) == -1 and int(x.min()) == -1 for x in tail.split(2 ** 29))


def test_append_of_as_many_tokens_as_32_bits_count():
    n = 2 ** 31 - 1
    slots = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    slots[-1] = 17
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV).expand(n, 1, 64)
    k, v = (torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((2, 1), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    M.KVCache(k, v, ks, vs).append(x, x, slots)
    assert not k[0].any() and not k[1, 0, 2:].any() and k[1, 0, 1].all()


def test_an_empty_free_list_serves_rows_that_need_no_block():
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    table = base._dev([[4], [9]])
    p = M.kv_plan(base._dev([3, 16]), base._dev([2, 1]), table, none, base._dev([0]), 16, 3)
    assert base._np(p.slot_map).tolist() == [67, 68, -1] and int(p.n_unserved) == 1
    seq, n = base._dev([3, 16]), base._dev([0])
    M.kv_release(torch.tensor([True, False], device=DEV), seq, table, none, n, 16)
    assert base._np(seq).tolist() == [0, 16] and int(n) == 0


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("around", [-60.0, -40.0, -20.0, -14.0, -9.0])
@pytest.mark.parametrize("experts,k", [(256, 32), (60, 32), (896, 16)])
def test_route_orders_neighbouring_logits(experts, k, around, scoring):
    """Consecutive fp32 logits, whose scores differ by 8 of their own last places or more: more
    than the exponentials (2 each) and the reciprocals (1 each) may be off together."""
    step = np.spacing(np.float32(abs(around)))
    rng = np.random.default_rng(experts)
    x = np.float32(around) + np.arange(experts) * np.float64(step)
    x = rng.permuted(np.tile(x, (50, 1)), axis=1).astype(np.float32)
    assert len(np.unique(x[0])) == experts
    if scoring == "softmax":
        x[:, 0] = 0.0                               # the row's largest: the others subtract exactly
    want_i, _ = ref.route(x.astype(np.float64), None, k, scoring, 1, 1, 1, True, 1.0)
    idx, w = M.moe_route(base._dev(x, torch.float32), k, scoring=scoring)
    assert np.array_equal(base._np(idx), want_i)
    assert (w[:, :-1] >= w[:, 1:]).all()


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_route_writes_the_scores_it_compared(scoring):
    """Without a bias the written scores descend, equal ones by ascending expert."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(20000, 896, generator=g, device=DEV) * 4
    idx, w = M.moe_route(x, 32, scoring=scoring, renormalize=False)
    a, b = w[:, :-1], w[:, 1:]
    assert (a >= b).all()
    assert (idx[:, :-1] < idx[:, 1:])[a == b].all()


# ---------------------------------------------------------------------------
# First calls
# ---------------------------------------------------------------------------
FIRST_CALLS = """
import sys
sys.path[:0] = {path!r}
import threading, torch
import moe_decode_step_gb300 as M
torch.cuda.init()
lib, n = M.lib(), 16
gate, got = threading.Barrier(n), [None] * n
def first(i):
    torch.cuda.set_device(0)
    gate.wait()
    got[i] = lib.moe_kv_attention_workspace(128)
threads = [threading.Thread(target=first, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
assert min(got) > 0 and len(set(got)) == 1, got
"""


def test_first_calls_of_many_threads_agree():
    import subprocess
    import sys
    p = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(path=sys.path)],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


# ---------------------------------------------------------------------------
# Rows that shrink
# ---------------------------------------------------------------------------
def _conserved(table, seq, free, n, bs, n_blocks):
    """Every block is held by one row or free, once."""
    held = [int(b) for r in range(len(seq)) for b in table[r, :-(-int(seq[r]) // bs)]]
    ids = held + [int(b) for b in free[:n]]
    assert sorted(ids) == list(range(n_blocks))


def test_rejected_drafts_give_their_blocks_back():
    """Steps of eight drafts of which some are accepted, for as many steps as would use up a
    stack that lost a block in each."""
    bs, rows, n_blocks, mb = 16, 5, 40, 8
    rng = np.random.default_rng(0)
    table = torch.zeros(rows, mb, dtype=torch.int32, device=DEV)
    free = torch.arange(n_blocks, dtype=torch.int32, device=DEV)
    n, ctx = base._dev([n_blocks]), torch.zeros(rows, dtype=torch.int32, device=DEV)
    q = torch.full((rows,), 8, dtype=torch.int32, device=DEV)
    done = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for step in range(60):
        p = M.kv_plan(ctx, q, table, free, n, bs, 8 * rows)
        assert int(p.n_unserved) == 0
        n.copy_(p.n_free)
        keep = base._dev(base._np(ctx) + rng.integers(1, 9, rows))
        if step % 12 == 11:
            done[step // 12] = True
        M.kv_release(done, p.seq_lens, table, free, n, bs, keep_lens=keep)
        want = np.where(base._np(done), 0, base._np(keep))
        assert np.array_equal(base._np(p.seq_lens), want)
        _conserved(base._np(table), want, base._np(free), int(n), bs, n_blocks)
        ctx = torch.where(done | (p.seq_lens > 110), 0, p.seq_lens).to(torch.int32)
        if (p.seq_lens > 110).any():      # finished
            M.kv_release(p.seq_lens > 110, p.seq_lens, table, free, n, bs)
        done[:] = False


@pytest.mark.parametrize("rows", [1, 7, 600, 3000])
def test_release_past_kept_lengths_matches_row_by_row(rows):
    rng = np.random.default_rng(rows)
    bs, mb = 16, 6
    seq = rng.integers(0, bs * mb + 1, rows)
    keep = np.where(rng.random(rows) < 0.7, seq - rng.integers(0, 40, rows), rng.integers(-5, 200, rows))
    fin = rng.random(rows) < 0.2
    table = rng.permutation(rows * mb).reshape(rows, mb)
    free = np.concatenate([[7, 8, 9], np.full(rows * mb, -1)])
    want, lens = [7, 8, 9], seq.copy()
    for r in range(rows):
        k = 0 if fin[r] else int(keep[r])
        if k < 0 or k >= seq[r]:          # nothing past it
            continue
        want += table[r, -(-k // bs):-(-int(seq[r]) // bs)].tolist()
        lens[r] = k
    t_seq, t_free, t_n = base._dev(seq), base._dev(free), base._dev([3])
    M.kv_release(torch.from_numpy(fin).to(DEV), t_seq, base._dev(table), t_free, t_n, bs,
                 keep_lens=base._dev(keep))
    assert np.array_equal(base._np(t_seq), lens)
    assert int(t_n) == len(want) and base._np(t_free)[:len(want)].tolist() == want
    with pytest.raises(ValueError, match="keep_lens"):
        M.kv_release(torch.from_numpy(fin).to(DEV), t_seq, base._dev(table), t_free, t_n, bs,
                     keep_lens=base._dev(keep).long())


# ---------------------------------------------------------------------------
# Append: skipped tokens
# ---------------------------------------------------------------------------
def _expect_append(codes, scale, new, slots, bs):
    """As moe_kv_append states it: the tokens of a block are those among the slot map's entries,
    whatever skipped ones lie between."""
    codes, scale = codes.copy(), scale.copy()
    n_blocks, hkv = scale.shape
    for b in dict.fromkeys(int(s) // bs for s in slots if 0 <= s < n_blocks * bs):
        ts = [t for t, s in enumerate(slots) if s >= 0 and s // bs == b]
        offs = [int(slots[t]) % bs for t in ts]
        for h in range(hkv):
            e = ref.block_exp(np.abs(new[ts, h]).max())
            if offs[0]:
                old = int(np.clip(int(scale[b, h]) - 127, -60, 60))
                if old < e:
                    codes[b, h, :offs[0]] = ref.e4m3_round(
                        ref.e4m3_table()[codes[b, h, :offs[0]]] * 2.0 ** (old - e))
                e = max(e, old)
            scale[b, h] = e + 127
            codes[b, h, offs] = ref.e4m3_round(new[ts, h] * 2.0 ** -e)
    return codes, scale


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bs", [16, 64, 128])
def test_append_with_skipped_tokens_inside_blocks(bs, many):
    """Tokens that go nowhere between those of one block, few and long runs of them, at chunks'
    ends and at the map's: still one scale a block, whatever order the GPU works in."""
    rng = np.random.default_rng(bs + many)
    lens = [(0, 3 * bs), (bs - 3, 40), (7, 1), (0, 1), (5, 2), (bs // 2, 2 * bs + 9), (1, bs - 1)]
    lens = lens * (5 if many else 1) + ([(3, 1500)] if many else [])
    need = [-(-(c + n) // bs) for c, n in lens]
    n_blocks, d, hkv = sum(need) + 1, 128, 2
    ids = rng.permutation(n_blocks)
    slots, at = [], 0
    for (c, n), k in zip(lens, need):
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(c, c + n)]
        at += k
    slots = np.array(slots)
    skip = rng.random(len(slots)) < 0.2
    for a, n in ((3, 2), (bs + 1, bs - 3), (60, 10), (len(slots) - 2, 2)):
        skip[a:a + n] = True
    slots[skip] = rng.choice([-1, n_blocks * bs, 2 ** 31 - 1], int(skip.sum()))
    codes = rng.integers(0, 127, (2, n_blocks, hkv, bs, d)).astype(np.uint8)
    scale = rng.integers(127 - 14, 127 - 3, (2, n_blocks, hkv)).astype(np.uint8)
    new = rng.standard_normal((2, len(slots), hkv, d)) * 2.0 ** rng.integers(-6, 4, (2, len(slots), 1, 1))
    t = [torch.from_numpy(x).to(torch.bfloat16).to(DEV) for x in new]
    for _ in range(3):
        k, v = torch.from_numpy(codes).to(DEV)
        ks, vs = torch.from_numpy(scale).to(DEV)
        M.KVCache(k, v, ks, vs).append(t[0], t[1], base._dev(slots))
        for s, (c, sc) in enumerate(((k, ks), (v, vs))):
            wc, ws = _expect_append(codes[s], scale[s], base._np(t[s].double()), slots, bs)
            assert np.array_equal(base._np(sc), ws), s
            assert np.array_equal(base._np(c), wc), s
