"""What no row sees has no part in any row: unwritten tokens may hold anything (infinite and NaN scales and offsets, large
finite ones), new tokens whose bit no row has and tokens before every row's window among them.

The results have to be the same bits whatever the unseen tokens hold, and within the tolerances of test_kv4_gpu.py and
test_kv4_tree_gpu.py, derived there.
"""
import numpy as np
import pytest

import kv_ref
import tree_ref
from test_kv4_gpu import _built, close, make  # noqa: F401
from test_kv4_tree_gpu import near

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN, TOP, ONE = 0x7C00, 0x7E00, 0x7BFF, 0x3C00
# (ks, ko, vs, vo) as fp16 bits
GARBAGE = [(INF,) * 4, (NAN,) * 4, (TOP,) * 4, (ONE, ONE, ONE, INF), (ONE, ONE, ONE, NAN), (ONE, ONE, INF, ONE), (ONE, ONE, TOP, 0),
           (INF, ONE, ONE, ONE), (ONE, 0xFC00, 0xFBFF, 0xFC00)]


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def overwrite(cache, table, positions, params, seed=0):
    """Random codes, and these scales and offsets, for positions of a request, every head."""
    rng = np.random.default_rng(seed)
    D, page = cache.head_dim, cache.page_size
    raw = cache.buf.cpu().numpy().reshape(cache.n_pages, cache.kv_heads, page // 16, 16 * (D + 8))
    for t in positions:
        granule = raw[table[t // page], :, t % page // 16]
        i = t % 16
        granule[:, i * (D // 2):(i + 1) * (D // 2)] = rng.integers(0, 256, (cache.kv_heads, D // 2))
        granule[:, 16 * D + 8 * i:16 * D + 8 * i + 8] = np.array(params, np.uint16).view(np.uint8)
    cache.buf.copy_(cuda(raw.reshape(-1)))


CASES = [
    # lens, nq, hq, hkv, D, page, window
    ([90], [6], 2, 2, 128, 16, 0),             # up to 16 rows a key head
    ([200], [5], 8, 2, 64, 16, 40),
    ([200], [3], 16, 1, 128, 32, 70),          # 48
    ([150], [40], 4, 1, 128, 16, 0),           # many
    ([300], [30], 8, 1, 64, 48, 75),
    ([400], [33], 8, 2, 128, 64, 130),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", CASES)
def test_trees(lens, nq, hq, hkv, D, page, window):
    import w4a16_mixed_precision_gb300 as w4
    n, first = nq[0], lens[0] - nq[0]
    rng = np.random.default_rng(lens[0])
    see = tree_ref.sees(tree_ref.random_parents(n, rng))
    gone = [1, n // 2, n - 2]           # new tokens that no row sees
    see[:, gone] = False
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=lens[0])
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q, tree = cuda(rng.standard_normal((n, hq, D)).astype(np.float16)), cuda(tree_ref.bits(see, -(-n // 32)))
    lo = max(0, first + int(see.sum(1).min()) - window) if window else 0
    unseen = list(range(lo)) + [first + j for j in gone]
    y = w4.kv4_tree_attention(q, cache, batch, tree, ws, window=window)
    ref = tree_ref.attention(q.cpu().numpy(), kv_ref.values(k), kv_ref.values(v), see, D ** -0.5, window)
    near(y.cpu().numpy(), ref, kv_ref.values(v), n * hq // hkv)
    for params in GARBAGE:
        overwrite(cache, batch.page_table[0].tolist(), unseen, params)
        assert torch.equal(w4.kv4_tree_attention(q, cache, batch, tree, ws, window=window), y), [hex(x) for x in params]
    assert w4.device_status(ws) == 0


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", [([200], [2], 4, 2, 128, 16, 70), ([300], [100], 4, 2, 128, 16, 75),
                                                          ([700], [66], 2, 2, 64, 64, 130)])
def test_runs_under_a_window(lens, nq, hq, hkv, D, page, window):
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=lens[0] + 1)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q = cuda(np.random.default_rng(lens[0]).standard_normal((nq[0], hq, D)).astype(np.float16))
    y = w4.kv4_attention(q, cache, batch, ws, window=window)
    close(y.cpu().numpy(), kv_ref.attention(q.cpu().numpy(), kv_ref.values(k), kv_ref.values(v), nq[0], D ** -0.5, window),
          kv_ref.values(v))
    for params in GARBAGE:
        overwrite(cache, batch.page_table[0].tolist(), range(lens[0] - nq[0] - window + 1), params)
        assert torch.equal(w4.kv4_attention(q, cache, batch, ws, window=window), y), [hex(x) for x in params]
    assert w4.device_status(ws) == 0
