"""kv_ref and tree_ref for long caches: the same in torch, on the GPU (nothing of the package's)."""
from __future__ import annotations

import torch


def quantise(x):
    """fp16 vectors [..., D] -> their codes less 8, scales and offsets, all in 64 bits: what kv_ref.quantise does."""
    f = x.float()
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).half().float()
    o = (lo + 8 * s).half().float()
    c = torch.where(s > 0, torch.round((f - o) / s).clamp(-8, 7), torch.zeros_like(f))
    return c.double(), s.double(), o.double()


def values(x):
    c, s, o = quantise(x)
    return s * c + o


def attention(q, k, v, see, scale, window=0, rounded=False):
    """One request: q fp16 [n, Hq, D], k, v fp16 [len, Hkv, D], see bool [n, n] among the new tokens -> [n, Hq, D] in 64
    bits.  rounded: every probability times its value's scale is rounded to fp16 first, at a magnitude where fp16 has
    all its bits, and nothing else."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    first, group = length - n, hq // hkv
    hide = torch.zeros((n, length), dtype=torch.bool, device=q.device)
    hide[:, first:] = ~see
    if window:
        at = torch.arange(length, device=q.device)
        hide |= (at < first) & (at < (first + see.sum(1) - window)[:, None])
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for h in range(hkv):
        kk, (c, s, o) = values(k[:, h]), quantise(v[:, h])
        for g in range(h * group, (h + 1) * group):
            x = (q[:, g].double() @ kk.t() * scale).masked_fill(hide, -torch.inf)
            p = (x - x.amax(-1, keepdim=True).clamp(min=-1e300)).exp()
            ps = p * s[:, 0]
            if rounded:  # the largest below 2^14
                unit = torch.exp2(13 - torch.floor(torch.log2(ps.amax(-1, keepdim=True).clamp(min=1e-300))))
                ps = (ps * unit).half().double() / unit
            total = p.sum(-1, keepdim=True)
            out[:, g] = torch.where(total > 0, (ps @ c + p @ o) / total.clamp(min=1e-300), torch.zeros_like(total))
    return out


def rms(x):
    return float((x.double() ** 2).mean().sqrt())
