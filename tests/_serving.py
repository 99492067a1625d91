"""Plain 64-bit restatements of the serving operators, and the inputs their
tests share.  Everything here runs on the CPU in float64 numpy."""
import numpy as np

E4M3 = None


def e4m3_table():
    """Value of every E4M3 code (OFP8 E4M3FN): bias 7, no infinities, S.1111.111 NaN."""
    global E4M3
    if E4M3 is None:
        c = np.arange(256)
        e, m = (c >> 3) & 15, c & 7
        v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
        v[(c & 127) == 127] = np.nan
        E4M3 = np.where(c & 128, -v, v)
    return E4M3


def e4m3_round(x):
    """Codes of the nearest E4M3 values (ties to the even code; past 448, infinities
    too, to 448; NaN to NaN) of float64 x, by search in the table."""
    tab = e4m3_table()[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(tab, a), 1, 126)
    lo = hi - 1
    dl, dh = a - tab[lo], tab[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def block_exp(amax):
    """Smallest integer e in [-60, 60] with amax <= 448 * 2^e."""
    e = -60
    while e < 60 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def read_cache(codes, scale):
    """[n_blocks, heads, block, dim] values of codes and scale bytes (uint8)."""
    e = np.clip(scale.astype(int) - 127, -60, 60)
    return e4m3_table()[codes] * 2.0 ** e[:, :, None, None]


def attention(q, k, v, table, seq_lens, q_start, scale, causal, window, n_blocks):
    """out, lse, A (the same average of |v|), S (largest sum_d |q_d k_d| * scale over
    the seen keys) in float64; k, v from read_cache."""
    tokens, heads, d = q.shape
    hkv, bs = k.shape[1], k.shape[2]
    out = np.zeros((tokens, heads, d))
    mag = np.zeros_like(out)
    lse = np.full((tokens, heads), -np.inf)
    span = np.zeros((tokens, heads))
    for r, seq in enumerate(seq_lens):
        a, b = q_start[r], q_start[r + 1]
        j = np.arange(seq)
        ids = table[r, j // bs]
        ok = (ids >= 0) & (ids < n_blocks)
        safe = np.where(ok, ids, 0)
        for i in range(b - a):
            p = seq - (b - a) + i
            see = ok & ((j <= p) if causal else True)
            if window:
                see = see & (j > p - window)
            js = j[see]
            if not len(js):
                continue
            for h in range(heads):
                kk = k[safe[js], h // (heads // hkv), js % bs]
                vv = v[safe[js], h // (heads // hkv), js % bs]
                s = kk @ q[a + i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                out[a + i, h] = w @ vv / z
                mag[a + i, h] = w @ np.abs(vv) / z
                lse[a + i, h] = m + np.log(z)
                span[a + i, h] = (np.abs(kk) @ np.abs(q[a + i, h])).max() * scale
    return out, lse, mag, span


def plan(ctx, q, table, free, n_free, bs, n_slots):
    """Row by row, as moe_kv_plan states it; returns the outputs and the new table."""
    table = table.copy()
    rows, mb = table.shape
    seq, q_start, slot = [], [0], np.full(n_slots, -1, np.int64)
    want = used = unserved = 0
    for r in range(rows):
        c, n = int(ctx[r]), int(q[r])
        ok = c >= 0 and n >= 0
        if not ok:
            c, n = max(c, 0), 0
        first = q_start[-1]
        q_start.append(first + n)
        have, total = -(-c // bs), -(-(c + n) // bs)
        if ok and total > mb:
            ok = False
        elif ok:
            want += total - have
            ok = (total == have or want <= n_free) and (n == 0 or first + n <= n_slots)
        if not ok:
            unserved += 1
            seq.append(c)
            continue
        for b in range(have, total):
            table[r, b] = free[n_free - 1 - (want - total + b)]
        if total > have:
            used = want
        seq.append(c + n)
        for i in range(n):
            pos = c + i
            slot[first + i] = table[r, pos // bs] * bs + pos % bs
    return np.array(seq), np.array(q_start), slot, n_free - used, unserved, table


def route(logits, bias, k, scoring, groups, topk_groups, group_top, renorm, scale):
    """idx, w per row; logits float64 holding the values the call gets."""
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-logits))
        else:
            m = np.fmax.reduce(logits, axis=1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            e = np.exp(logits - m)
            z = e.sum(axis=1, keepdims=True)
            s = np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))
    sel = s + (0.0 if bias is None else bias)
    rows, n = sel.shape
    idx = np.zeros((rows, k), int)
    w = np.zeros((rows, k))
    size = n // groups
    for r in range(rows):
        key = [(-v if v == v else np.inf) for v in sel[r]]
        left = range(n)
        if groups > 1:
            gk = []
            for g in range(groups):
                best = sorted(key[g * size:(g + 1) * size])[:group_top]
                gk.append((sum(best), g))
            keep = sorted(gk)[:topk_groups]
            left = [e for _, g in keep for e in range(g * size, (g + 1) * size)]
        order = sorted(left, key=lambda e: (key[e], e))[:k]
        idx[r] = order
        p = s[r, order]
        if renorm:
            p = p / p.sum() if p.sum() != 0 else np.zeros(k)
        w[r] = scale * p
    return idx, w
