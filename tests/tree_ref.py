"""Plain implementations, in 64 bits, of what the operators for drafted trees compute (nothing of the package's)."""
from __future__ import annotations

import numpy as np


def random_parents(n, rng, back=6):
    return np.array([-1 if i == 0 or rng.random() < 0.05 else max(0, i - 1 - int(rng.integers(0, back))) for i in range(n)],
                    np.int32)


def sees(parents):
    """bool [n, n]: the token itself and its ancestors."""
    n = len(parents)
    out = np.eye(n, dtype=bool)
    for i in range(n):
        if parents[i] >= 0:
            out[i] |= out[parents[i]]
    return out


def bits(see, words):
    """bool [n, m] -> int32 [n, words]."""
    n, m = see.shape
    full = np.zeros((n, words * 32), bool)
    full[:, :min(m, words * 32)] = see[:, :words * 32]
    return (full.reshape(n, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def attention(q, k, v, see, scale, window=0):
    """One request: q [n, Hq, D], k, v [len, Hkv, D], see bool [n, n] among the new tokens -> [n, Hq, D].  Masked tokens
    do not enter, whatever they hold; a row that sees nothing is zero."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    g, first = hq // hkv, length - n
    out = np.zeros((n, hq, d))
    for i in range(n):
        lo = max(0, first + int(see[i].sum()) - window) if window else 0
        at = np.concatenate([np.arange(lo, first), first + np.flatnonzero(see[i])])
        if not at.size:
            continue
        for h in range(hq):
            kk, vv = k[at, h // g], v[at, h // g]
            s = kk @ q[i, h].astype(np.float64) * scale
            with np.errstate(all="ignore"):
                p = np.exp(s - s.max())
                out[i, h] = p @ vv / p.sum()
    return out


def rotate(x, positions, cos, sin, axes, interleaved):
    """x fp16 [T, H, D], positions [axes, T], cos, sin fp32 [rows, rot / 2], axes [rot / 2] -> the rotated channels as
    fp32 products and sums rounded one by one give them, rounded to fp16, and in 64 bits."""
    out32, out64 = x.astype(np.float32), x.astype(np.float64)
    half = cos.shape[1]
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        at = positions[axes[j]]
        for out, t in ((out32, np.float32), (out64, np.float64)):
            c, s = cos[at, j].astype(t)[:, None], sin[at, j].astype(t)[:, None]
            x1, x2 = x[..., a].astype(t), x[..., b].astype(t)
            with np.errstate(all="ignore"):
                out[..., a], out[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    with np.errstate(all="ignore"):
        return out32.astype(np.float16), out64
