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
