"""Plain implementations of the 4-bit cache's format and of attention over it, in
64 bits, for the tests (nothing of the package's)."""
from __future__ import annotations

import numpy as np


def quantise(x):
    """fp16 vectors [..., D] -> the fp16 values the format stands for (fp32
    arithmetic as the format defines it) and the codes."""
    x = np.asarray(x, np.float16).astype(np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        s = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16).astype(np.float32)
        o = (lo + np.float32(8) * s).astype(np.float16).astype(np.float32)
        c = np.where(s > 0, np.clip(np.rint((x - o) / np.where(s > 0, s, np.float32(1))), -8, 7), np.float32(0))
    v = s.astype(np.float64) * c + o
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    return np.where(bad, np.nan, v), c


def values(x):
    """The values in 64 bits (exact: attention works on these, not on their fp16 roundings)."""
    return quantise(x)[0]


def attention(q, k, v, n_new, scale, window=0):
    """One request in 64 bits: q [n_new, Hq, D], k, v [len, Hkv, D] -> [n_new, Hq, D].  Masked keys do
    not enter, whatever they hold; a row that sees nothing is zero."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    g = hq // hkv
    out = np.zeros((n, hq, d))
    for i in range(n):
        pos = length - n_new + i
        lo = max(0, pos - window + 1) if window else 0
        if pos < 0:
            continue
        for h in range(hq):
            kk, vv = k[lo:pos + 1, h // g], v[lo:pos + 1, h // g]
            s = kk @ q[i, h].astype(np.float64) * scale
            with np.errstate(all="ignore"):
                p = np.exp(s - s.max())
                out[i, h] = p @ vv / p.sum()
    return out
