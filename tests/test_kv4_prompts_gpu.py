"""Prompt attention where a CTA's stripe runs through several items (256 query rows of a key head
each), and where value vectors have a scale of zero, against the formula in 64 bits.

Tolerances are those of test_kv4_gpu.py, derived there.
"""
import numpy as np
import pytest

import kv_ref
from test_kv4_gpu import _built, close, make, split  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def exact(q, k, v, scale, window=0):
    """kv_ref.attention's formula for the last rows of one request, head by head in 64 bits on the GPU."""
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().double()  # noqa: E731
    q, k, v = cu(q), cu(k), cu(v)
    n, hq, _ = q.shape
    length, hkv, _ = k.shape
    pos = torch.arange(length - n, length, device="cuda")[:, None]
    t = torch.arange(length, device="cuda")
    hide = t > pos
    if window:
        hide = hide | (t + window <= pos)
    out = torch.empty_like(q)
    for h in range(hq):
        s = (q[:, h] @ k[:, h // (hq // hkv)].t() * scale).masked_fill(hide, -float("inf"))
        out[:, h] = torch.softmax(s, -1) @ v[:, h // (hq // hkv)]
    return out.cpu().numpy()


STRIPES = [
    # lens, nq, hq, hkv, D, page, window
    ([4400], [1000], 40, 40, 128, 64, 0),       # more long items than SMs, about one a stripe: most stripes cross an end
    ([4400], [1000], 24, 24, 128, 32, 0),       # fewer items than SMs, each cut in two or three
    ([3800, 4100], [350, 350], 64, 8, 128, 16, 0),
    ([4400], [1000], 40, 40, 64, 64, 0),
    ([6000], [1000], 24, 24, 128, 128, 4000),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", STRIPES)
def test_stripes_through_several_items(lens, nq, hq, hkv, D, page, window):
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=sum(lens) + hq)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = np.random.default_rng(50).standard_normal((sum(nq), hq, D)).astype(np.float16)
    dq = torch.from_numpy(q).cuda()
    y = w4.kv4_attention(dq, cache, batch, ws, window=window)
    for _ in range(20):
        assert torch.equal(w4.kv4_attention(dq, cache, batch, ws, window=window), y)
    assert w4.device_status(ws) == 0
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
        close(yy, exact(qq, kv[b], vv[b], D ** -0.5, window), vv[b])


@pytest.mark.parametrize("far", [12, 84, 200])
@pytest.mark.parametrize("kind", ["zero", "constant", "all"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq", [1, 80])
def test_constant_values_with_large_scores(nq, D, kind, far):
    """A value vector whose channels are all equal has a scale of 0, so its probability enters no product with
    codes: a score far above the earlier ones (by `far` nats) must move a row's reference all the same.
    Tolerance: as in test_kv4_gpu.py, and 2^-20 of a score's products' magnitudes (fp32 sums of them, 2^-24
    each) on either of two scores."""
    import w4a16_mixed_precision_gb300 as w4
    lens, hq, hkv, page = [400], 4, 2, 16
    k, v, cache, batch, hist = make(lens, [nq], hkv, D, page, seed=60)
    # every query has 1 in its last channel beside small numbers; keys have 0 there but for a few tokens
    q = (0.05 * np.random.default_rng(61).standard_normal((nq, hq, D))).astype(np.float16)
    q[:, :, D - 1] = 1
    k *= np.float16(0.5)
    k[:, :, D - 1] = 0
    lifted = [200, 231, 257, 300, 301, 302, 303]
    k[lifted, :, D - 1] = np.float16(far)
    k[302, :, D - 1] = np.float16(far + 1)
    v[lifted] = np.float16(0 if kind == "zero" else 0.75)
    v[303] = np.float16(-1.5)
    if kind == "all":
        v[:] = (np.arange(400) % 7 - 3).astype(np.float16)[:, None, None] * np.float16(0.25)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws, scale=1.0).cpu().numpy().astype(np.float64)
    assert w4.device_status(ws) == 0
    vals = kv_ref.values(v)
    ref = exact(q, kv_ref.values(k), vals, 1.0)
    mag = np.abs(q.astype(np.float64)).sum(-1)[:, :, None] * 15 * np.abs(k.astype(np.float64)).max()
    tol = 2.0 ** -11 * np.abs(ref) + (2.0 ** -12 + 2.0 ** -20 * mag) * np.abs(vals).max() + 2.0 ** -24
    assert (np.abs(y - ref) <= tol).all()   # NaN fails too


@pytest.mark.parametrize("window", [2**31 - 1, 2**30, 18])
@pytest.mark.parametrize("length,nq", [(2, 5), (20, 23), (100, 164)])
def test_largest_windows_and_more_new_tokens_than_the_length(length, nq, window):
    """A window that hides nothing, up to the largest number, leaves the rows that see tokens as they are,
    in a request whose first new tokens have negative positions too."""
    import w4a16_mixed_precision_gb300 as w4
    hq, hkv, D, page = 4, 2, 64, 16
    k, v, cache, batch, hist = make([length], [length], hkv, D, page, seed=70)
    ws = w4.Kv4Workspace(w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, nq, nq), hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = np.random.default_rng(71).standard_normal((nq, hq, D)).astype(np.float16)
    start = torch.tensor([0, nq], dtype=torch.int32, device="cuda")
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, w4.Kv4Batch(batch.page_table, batch.lengths, start, nq, nq),
                         ws, window=window).cpu().numpy()
    assert w4.device_status(ws) == 7   # MARLIN_ERR_BOUNDS: reported
    none = nq - length
    assert (y[:none] == 0).all()
    close(y[none:], kv_ref.attention(q[none:], kv_ref.values(k), kv_ref.values(v), length, D ** -0.5,
                                     window if window < length else 0), kv_ref.values(v))
