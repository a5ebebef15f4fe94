"""Plain 64-bit references of the int8 rows, the int8 product, the beam selection and
the state reordering (numpy, no library code)."""
from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def quantize_rows(x):
    """(q int8, scale float32) of float64 rows: nearest integer to the exact quotient by
    the stored scale, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(1)
    a = np.abs(np.where(bad[:, None], 0.0, x)).max(1)
    scale = (a / 127.0).astype(np.float32)
    d = scale.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d[:, None] > 0, np.rint(np.where(bad[:, None], 0.0, x) / d[:, None]), 0.0)
    scale[bad] = np.nan
    return np.clip(q, -127, 127).astype(np.int8), scale


def product(xq, xs, wq, ws, bias=None):
    """(y, p): the product with and without the bias, float64."""
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T  # whole numbers below 2^53
    p = acc * ws.astype(np.float64)[None] * xs.astype(np.float64)[:, None]
    return (p if bias is None else p + bias.astype(np.float64)[None]), p


def product_tolerance(y, p, eps_out, tiny):
    """The int32 sum's conversion, the scales' product and the multiplication are off by
    half a float32 step each, the addition by half a step of its result; then one
    rounding to the output's type (none for float32), half its smallest step below."""
    half = 2.0 ** -24
    return 3.01 * half * np.abs(p) + 1.01 * (half + eps_out / 2) * np.abs(y) + tiny


def fused32(a, b, c):
    """a * b + c of float32 arrays rounded once to float32. The product is exact in float64
    (48 bits) and the sum's error is known exactly, so the sum is first rounded to odd: its
    last bit stands for all that was cut off, and 53 bits rounded to 24 then give what the
    exact sum would."""
    p, c = a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)
    bits = s.view(np.int64)
    away = (err > 0) == (s > 0)  # the exact sum is farther from zero than s
    odd = np.where((err != 0) & (bits & 1 == 0), np.where(away, bits + 1, bits - 1), bits)
    return odd.view(np.float64).astype(np.float32)


def beam_select(z, score, n, finished=None, length=None, eos=-1, alpha=0.0):
    """Selection over (B, W, V) float64 logits; returns a dict of (B, n) arrays."""
    B, W, V = z.shape
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), F32_MAX)
    out = {"token": np.full((B, n), -1), "parent": np.full((B, n), -1), "score": np.full((B, n), -np.inf),
           "finished": np.zeros((B, n), bool), "length": np.zeros((B, n), int)}
    for b in range(B):
        cand = []
        for w in range(W):
            cum = float(score[b, w])
            done = finished is not None and bool(finished[b, w])
            ln = 0 if length is None else int(length[b, w])
            new = ln if done else ln + 1
            if np.isnan(cum) or cum == -np.inf:
                continue
            over = float(max(new, 1)) ** alpha if alpha else 1.0
            if done:
                cand.append((-cum / over, w, 0.0, eos, cum, new, True))
                continue
            keep = np.flatnonzero(z[b, w] > -np.inf)
            if keep.size == 0:
                continue
            d = z[b, w][keep] - z[b, w][keep].max()
            logp = d - np.log(np.exp(d).sum())
            for i in np.lexsort((keep, -d))[:n]:
                s = cum + logp[i]
                cand.append((-s / over, w, -d[i], int(keep[i]), s, new, int(keep[i]) == eos))
        cand.sort()
        for j, (_, w, _, v, s, new, fin) in enumerate(cand[:n]):
            out["token"][b, j], out["parent"][b, j], out["score"][b, j] = v, w, s
            out["finished"][b, j], out["length"][b, j] = fin, new
    return out


def reorder(state, parent, beams, before):
    """Rows of `before` (the result's buffer) replaced by their parents' rows of `state`."""
    B, n = parent.shape
    out = before.copy()
    for b in range(B):
        for j in range(n):
            if 0 <= parent[b, j] < beams:
                out[b * n + j] = state[b * beams + parent[b, j]]
    return out
