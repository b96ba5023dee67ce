"""Tree attention: a row is zero where it sees no token, not where its scores happen to be minus infinity.  Tolerances are
those of test_kv4_tree_gpu.py, derived there."""
import numpy as np
import pytest

import kv_ref
import tree_ref
from test_kv4_gpu import _built, make  # noqa: F401
from test_kv4_tree_gpu import near

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("nq,hq", [(4, 2), (5, 8), (40, 4)])
@pytest.mark.parametrize("before", [0, 100])
def test_scores_of_minus_infinity_are_not_an_empty_row(nq, hq, before):
    """Keys above zero and a query with minus infinity: every score is minus infinity and the softmax undefined, as for
    kv4_attention.  Rows that see nothing are zero whatever their query holds."""
    import w4a16_mixed_precision_gb300 as w4
    D, length = 128, before + nq
    k, v, cache, batch, hist = make([length], [nq], 1, D, 16, seed=nq)
    rng = np.random.default_rng(nq)
    k[:] = rng.uniform(0.5, 1.0, k.shape)
    k[..., 7] = 2                      # the largest code of every key
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q = rng.standard_normal((nq, hq, D)).astype(np.float16)
    q[1, 1, 7] = q[3, 0, 7] = -np.inf
    see = tree_ref.sees(tree_ref.random_parents(nq, rng))
    see[3] = False
    y = w4.kv4_tree_attention(cuda(q), cache, batch, cuda(tree_ref.bits(see, -(-nq // 32))), ws).cpu().numpy()
    assert w4.device_status(ws) == 0
    with np.errstate(all="ignore"):
        ref = tree_ref.attention(q, kv_ref.values(k), kv_ref.values(v), see, D ** -0.5)
    assert np.isnan(ref[1, 1]).all() and np.isnan(ref[3, 0]).all() == (before > 0)
    near(y, ref, kv_ref.values(v), nq * hq)
    if not before:
        assert not y[3].any()


@pytest.mark.parametrize("lens,nq,hq,hkv,D", [
    ([5000], [40], 2, 1, 128),                                        # stripes cut the item: its parts are joined
    ([64 * (57 + 29 * i % 60) for i in range(40)], [9] * 40, 64, 8, 64),   # items that end inside a stripe after several pieces
    ([300, 200], [90, 75], 2, 2, 128),                                # a CTA each
])
def test_scores_of_minus_infinity_over_long_caches(lens, nq, hq, hkv, D):
    import w4a16_mixed_precision_gb300 as w4
    import kv_torch
    from test_kv4_tree_pieces_gpu import inputs
    q, k, v, cache, batch, ws, see, tree = inputs(lens, nq, hq, hkv, D, 64, 7)
    k.uniform_(0.5, 1.0)
    k[..., 7] = 2
    start = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    w4.kv4_append(k, v, cache, w4.Kv4Batch(batch.page_table, batch.lengths, start, sum(lens), max(lens)), ws)
    gone = torch.zeros((sum(nq), hq), dtype=torch.bool, device="cuda")
    gone[::5, ::3] = True
    q[..., 7][gone] = -float("inf")
    y = w4.kv4_tree_attention(q, cache, batch, tree, ws)
    assert w4.device_status(ws) == 0
    assert torch.equal(y.isnan().all(-1), gone) and torch.equal(y.isnan().any(-1), gone)
    t = h = 0
    for length, n, s in zip(lens, nq, see):
        clean = torch.where(gone[t:t + n, :, None], torch.zeros_like(q[t:t + n]), q[t:t + n])
        ref = kv_torch.attention(clean, k[h:h + length], v[h:h + length], cuda(s), D ** -0.5)
        some = ~gone[t:t + n]
        near(y[t:t + n][some].cpu().numpy(), ref[some].cpu().numpy(), kv_torch.values(v[h:h + length]).cpu().numpy(), n * hq // hkv)
        t, h = t + n, h + length


@pytest.mark.parametrize("n,hq,window", [(3000, 1, 0), (700, 4, 5), (2000, 2, 0)])
def test_empty_rows_among_many(n, hq, window):
    """Nothing before the new tokens: rows without bits are zero, wherever stripes cut, even with a query of infinities."""
    import w4a16_mixed_precision_gb300 as w4
    import kv_torch
    D = 128
    k, v, cache, batch, hist = make([n], [n], 1, D, 64, seed=n)
    ws = w4.Kv4Workspace(batch, hq, cache)
    k, v = cuda(k), cuda(v)
    w4.kv4_append(k, v, cache, hist, ws)
    rng = np.random.default_rng(n)
    see = rng.random((n, n)) < 0.004
    see[::7] = False
    see[n - 1] = True
    q = rng.standard_normal((n, hq, D)).astype(np.float16)
    q[::14] = np.inf
    empty = ~see.any(1)
    q[~empty] = np.where(np.isinf(q[~empty]), np.float16(1), q[~empty])
    y = w4.kv4_tree_attention(cuda(q), cache, batch, cuda(tree_ref.bits(see, -(-n // 32))), ws, window=window)
    assert w4.device_status(ws) == 0 and empty.sum() > n // 8
    assert not y.cpu().numpy()[empty].any()
    ref = kv_torch.attention(cuda(np.nan_to_num(q, posinf=1)), k, v, cuda(see), D ** -0.5, window)
    near(y.cpu().numpy()[~empty], ref.cpu().numpy()[~empty], kv_ref.values(v.cpu().numpy()), n * hq)
