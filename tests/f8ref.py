"""64-bit references of the block-scaled e4m3 rows and products, the selection of experts
and their combination, with the tolerances of their float32 steps. Plain numpy: used by
the CPU and the GPU tests."""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)
# the 127 values that are not negative, by code: 16 exponents (the first subnormal) of 8 values, less the NaN
HELD = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:-1])
VALUES = np.concatenate([HELD, [np.nan], -HELD, [np.nan]])  # of all 256 codes
BORDERS = (HELD[1:] + HELD[:-1]) / 2


def encode(v):
    """Codes of the e4m3 values nearest to v, ties to even, beyond +-448 clamped."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    i = np.searchsorted(BORDERS, a, side="left")
    tie = (i < 126) & (BORDERS[np.minimum(i, 125)] == a)
    i = np.where(tie & (i % 2 == 1), i + 1, i)
    return (i + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize_rows(h):
    """(codes (N, K), scale float32 (N, blocks)) of h (N, K) in float64 holding float32 values."""
    N, K = h.shape
    nb = -(-K // 128)
    codes, scale = np.zeros((N, K), np.uint8), np.zeros((N, nb), np.float32)
    for b in range(nb):
        x = h[:, 128 * b:128 * b + 128]
        top = np.abs(x).max(1)
        with np.errstate(over="ignore", under="ignore", invalid="ignore"):
            d = (top / 448.0).astype(np.float32)
        d[~np.isfinite(top)] = np.nan
        ok = d > 0
        codes[ok, 128 * b:128 * b + 128] = encode(x[ok] / d[ok].astype(np.float64)[:, None])
        scale[:, b] = d
    return codes, scale


def product(xc, xs, wc, ws, bias=None):
    """(y, float32 error, 8-bit sum error) of codes and scales, in float64: y[n, m] and
    bounds of what float32 sums of exact products, and the matrix cores' sums, may be off.

    float32: a block's 128 products are exact, their sum has at most 128 additions that
    round (or cut) by 2^-23 of at most sum |p|; the scales' product is off by 2^-24 and each of the
    nb multiply-adds, and the addition of the partial sums, by 2^-23 of at most the sum of the magnitudes.
    8 bits: eight products are aligned to the largest and lose what lies below 2^-13 of
    its power of two: at most 7 * 2^-13 of the largest of each eight."""
    K = xc.shape[1]
    nb = -(-K // 128)
    X, W = VALUES[xc], VALUES[wc]
    y = np.zeros((xc.shape[0], wc.shape[0]))
    mag = np.zeros_like(y)
    over = np.repeat(ws.astype(np.float64), 128, axis=0)[:wc.shape[0]]  # (M, nb)
    for b in range(nb):
        x, w = X[:, 128 * b:128 * b + 128], W[:, 128 * b:128 * b + 128]
        s = xs[:, b].astype(np.float64)[:, None] * over[:, b][None]
        y += (x @ w.T) * s
        mag += (np.abs(x) @ np.abs(w).T) * np.abs(s)
    cut = mag  # (the largest of each eight is at most their sum)
    if bias is not None:
        y = y + bias.astype(np.float64)
        mag = mag + np.abs(bias.astype(np.float64))
    return y, mag * (128 + 3 + nb + 16) * 2.0 ** -23, cut * 7 * 2.0 ** -13


def silu_gate(g, u):
    """g / (1 + exp(-g)) * u of float32 values, in float64."""
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def select(z, k, normalize, scale=1.0):
    """expert, weight (float64), position, row, offsets of logits z (N, E) in float64."""
    N, E = z.shape
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), F32_MAX)
    expert, position = np.full((N, k), -1, np.int32), np.full((N, k), -1, np.int32)
    weight = np.zeros((N, k))
    lists = [[] for _ in range(E)]
    for n in range(N):
        order = sorted((-z[n, e], e) for e in range(E) if z[n, e] > -np.inf)[:k]
        if not order:
            continue
        top = -order[0][0]
        p = [math.exp(-v - top) for v, _ in order]
        total = math.fsum(p) if normalize else math.fsum(math.exp(v - top) for v in z[n] if v > -np.inf)
        for j, (_, e) in enumerate(order):
            expert[n, j], weight[n, j] = e, scale * p[j] / total
            lists[e].append((n, j))
    row, offsets = np.full(N * k, -1, np.int32), np.zeros(E + 1, np.int32)
    r = 0
    for e in range(E):
        for n, j in lists[e]:
            row[r], position[n, j] = n, r
            r += 1
        offsets[e + 1] = r
    return expert, weight, position, row, offsets


def combine(y, position, weight, add=None):
    """(out, float32 error) in float64."""
    N, k = position.shape
    out = np.zeros((N, y.shape[1])) if add is None else add.astype(np.float64)
    mag = np.abs(out)
    for j in range(k):
        p = position[:, j]
        ok = (p >= 0) & (p < y.shape[0])
        t = y[p[ok]].astype(np.float64) * weight[ok, j].astype(np.float64)[:, None]
        out[ok] += t
        mag[ok] += np.abs(t)
    return out, mag * (k + 1) * 2.0 ** -24
