"""Plain 64-bit restatements of the 8-bit products, norms and expert operators, the
inputs their tests share and the bounds they are held to.  Everything here runs on
the CPU in float64 numpy.

Bounds, from the arithmetic, half a step per rounding (HALF: torch.finfo(t).eps / 2):
 - a product's sums are fp32: every K = 32 instruction is taken to be off by 4
   half steps (2^-22) of the sum of absolute terms S at most, (K / 32 + 2) 2^-22 S
   in all; products of codes are exact and scales are powers of two;
 - swiglu: silu' is below 1.1; the exponential is off by (2 + 1.16 |g|) ulp and
   the division by 2, (6 + 1.2 |g|) 2^-23 of the result in all;
 - the norm: z is one fp32 addition; the mean of squares is off by fewer than 64
   roundings, half of which reach the root; with the three products 64 2^-24;
 - a sum of k weighted rows is off by k + 1 roundings of the sum of absolute terms;
 - an 8-bit value is off by half a step, 2^-4 of itself (2^-10 of its scale among
   the smallest), beside what the value itself is off by, and its scale is the
   exact one unless the block's largest lies that near to a border.
"""
import numpy as np
import torch

import _serving as s

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# (below 2^-14 fp16 has steps of 2^-24: half of one is 2^-25, whatever the value)
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E2M1 = np.concatenate([E2M1, -E2M1])


def blocks(n):
    return -(-n // 128)


def block_exp(amax):
    """Smallest integer e in [-126, 120] with amax <= 448 * 2^e, elementwise."""
    amax = np.asarray(amax, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, amax, 1) / 448.0)), -126)
    e = np.where(amax > 448.0 * 2.0 ** e, e + 1, e)
    e = np.where(amax <= 448.0 * 2.0 ** (e - 1), e - 1, e)
    return np.clip(e, -126, 120).astype(int)


def finite_max(y, axis):
    return np.where(np.isfinite(y), np.abs(y), 0.0).max(axis=axis)


def row_exps(y):
    """Exponents [rows, blocks] of values [rows, d]."""
    rows, d = y.shape
    p = np.zeros((rows, blocks(d) * 128))
    p[:, :d] = y
    return block_exp(finite_max(p.reshape(rows, -1, 128), 2))


def quantize(y):
    """Codes and scale bytes (uint8) of values [rows, d]."""
    e = row_exps(y)
    unit = 2.0 ** np.repeat(e, 128, axis=1)[:, :y.shape[1]]
    return s.e4m3_round(y / unit), (e + 127).astype(np.uint8)


def pack(w):
    """Codes and scale bytes of weights [n, k]: a scale per 128 x 128."""
    n, k = w.shape
    p = np.zeros((blocks(n) * 128, blocks(k) * 128))
    p[:n, :k] = w
    e = block_exp(finite_max(p.reshape(blocks(n), 128, blocks(k), 128), (1, 3)))
    unit = 2.0 ** np.repeat(np.repeat(e, 128, 0), 128, 1)[:n, :k]
    return s.e4m3_round(w / unit), (e + 127).astype(np.uint8)


def row_values(codes, scales):
    return s.e4m3_table()[codes] * 2.0 ** (
        np.repeat(scales.astype(int), 128, axis=1)[:, :codes.shape[1]] - 127)


def weight_values(w, scales, mx):
    if mx:
        v = np.empty((w.shape[0], 2 * w.shape[1]))
        v[:, 0::2], v[:, 1::2] = E2M1[w & 15], E2M1[w >> 4]
        return v * 2.0 ** (np.repeat(scales.astype(int), 32, axis=1) - 127)
    unit = np.repeat(np.repeat(scales.astype(int), 128, 0), 128, 1)[:w.shape[0], :w.shape[1]]
    return s.e4m3_table()[w] * 2.0 ** (unit - 127)


def random_x(rng, rows, k):
    """Codes and scales of activations whose rows and channels differ."""
    v = rng.standard_normal((rows, k)) * np.exp(0.5 * rng.standard_normal((1, k)))
    return quantize(v * np.exp(rng.standard_normal((rows, 1))))


def random_w(rng, n, k, mx):
    if mx:
        return (rng.integers(0, 256, (n, k // 2), np.uint8),
                rng.integers(118, 123, (n, k // 32)).astype(np.uint8))
    return pack(rng.standard_normal((n, k)) * k ** -0.5 * np.exp(0.3 * rng.standard_normal((n, 1))))


def product(x, w):
    """Values and their bound before any rounding of the output."""
    k = x.shape[1]
    return x @ w.T, (k / 32 + 2) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T)


def swiglu(p, tol):
    n = p.shape[1] // 2
    g, u, dg, du = p[:, :n], p[:, n:], tol[:, :n], tol[:, n:]
    sig = 1.0 / (1.0 + np.exp(-g))
    h = g * sig * u
    off = 1.1 * dg * (np.abs(u) + du) + np.abs(g * sig) * du + (
        6 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(h)
    return h, off


def check_values(got, want, tol, dtype, what=""):
    """got (a tensor of dtype) within tol and its own rounding of want."""
    got = got.detach().float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    off = np.abs(got - want)[~nan]
    bound = (tol + np.maximum(HALF[dtype] * (np.abs(want) + tol), TINY[dtype]))[~nan]
    assert (off <= bound).all(), (what, float((off / bound).max()))


def check_codes(codes, scales, want, tol, what=""):
    """The 8-bit form of values that are within tol of want."""
    codes = codes.view(torch.uint8).cpu().numpy()
    e = scales.view(torch.uint8).cpu().numpy().astype(int) - 127
    assert codes.shape == want.shape and e.shape == (want.shape[0], blocks(want.shape[1])), what
    lo = row_exps(np.maximum(np.abs(want) - tol, 0))
    hi = row_exps(np.abs(want) + tol)
    assert ((e >= lo) & (e <= hi)).all(), (what, e[(e < lo) | (e > hi)])
    unit = 2.0 ** np.repeat(e, 128, axis=1)[:, :want.shape[1]]
    got = s.e4m3_table()[codes] * unit
    bound = tol + np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * unit) * (1 + 1e-9)
    off = np.abs(got - want)
    assert (off <= bound).all(), (what, float((off / bound).max()))


def dispatch(idx, experts):
    """offsets, rows, slots, entry by entry."""
    tokens, k = idx.shape
    by = [[] for _ in range(experts)]
    for t in range(tokens):
        for j in range(k):
            if 0 <= idx[t, j] < experts:
                by[idx[t, j]].append((t, j))
    rows = np.full(tokens * k, -1)
    slots = np.full((tokens, k), -1)
    for i, (t, j) in enumerate(c for b in by for c in b):
        rows[i] = t
        slots[t, j] = i
    return np.concatenate([[0], np.cumsum([len(b) for b in by])]), rows, slots
