"""How a window over the new tokens is said: by leaving their bits out.  Tolerances are those of test_kv4_tree_gpu.py,
derived there."""
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


@pytest.mark.parametrize("n,hq,window", [(40, 2, 9), (70, 8, 33), (6, 4, 1)])
def test_a_window_over_new_tokens_by_their_bits(n, hq, window):
    """A run longer than its window, the bits of tokens beyond it left out, is kv4_attention under that window."""
    import w4a16_mixed_precision_gb300 as w4
    D, length = 128, n + 150
    k, v, cache, batch, hist = make([length], [n], 1, D, 16, seed=n)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q = np.random.default_rng(n).standard_normal((n, hq, D)).astype(np.float16)
    i = np.arange(n)
    see = (i <= i[:, None]) & (i > i[:, None] - window)
    y = w4.kv4_tree_attention(cuda(q), cache, batch, cuda(tree_ref.bits(see, -(-n // 32))), ws, window=window)
    assert w4.device_status(ws) == 0
    near(y.cpu().numpy(), kv_ref.attention(q, kv_ref.values(k), kv_ref.values(v), n, D ** -0.5, window), kv_ref.values(v), n * hq)
