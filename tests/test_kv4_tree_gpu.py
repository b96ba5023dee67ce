"""Masks and positions of drafted trees, and attention of trees over the 4-bit cache, against plain implementations.

Tolerances are those of test_kv4_gpu.py, derived there, and where a request has more than 48 query rows per key
head one rounding more: that kernel rounds every p s (a probability times its value vector's scale) to fp16, by at
most 2^-11 of itself.  The result is sum p (s (c - 8) + o) / sum p over codes c from 0 to 15, so that it moves by at
most 2^-11 of the largest |s (c - 8)|, which is 8 s = 8/15 of the vector's range.
"""
import numpy as np
import pytest

import kv_ref
import tree_ref
from test_kv4_gpu import _built, close, make, split  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("nq", [[1], [2, 1, 5], [32, 33, 31], [64], [0, 65, 0, 7], [300, 1, 96], [1000]])
def test_masks_and_positions(nq):
    import w4a16_mixed_precision_gb300 as w4
    rng = np.random.default_rng(sum(nq))
    lens = [n + int(rng.integers(0, 1 << 20)) for n in nq]
    parents = [tree_ref.random_parents(n, rng) for n in nq]
    if nq[0] == 1000:
        parents[0] = np.arange(-1, 999, dtype=np.int32)  # a run of tokens
    start = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    batch = w4.Kv4Batch(torch.zeros((len(nq), 1), dtype=torch.int32, device="cuda"), cuda(np.array(lens, np.int32)),
                        cuda(start), sum(nq), max(nq))
    ws = w4.Kv4Workspace(batch, 1, w4.Kv4Cache(1, 1, 64, 16))
    mask, positions = w4.kv4_tree(cuda(np.concatenate(parents)), batch, ws)
    assert w4.device_status(ws) == 0
    words = -(-max(nq) // 32)
    assert mask.shape == (sum(nq), words) and mask.dtype == positions.dtype == torch.int32
    see = [tree_ref.sees(p) for p in parents]
    assert np.array_equal(mask.cpu().numpy(), np.concatenate([tree_ref.bits(s, words) for s in see]))
    assert np.array_equal(positions.cpu().numpy(), np.concatenate([n - len(s) + s.sum(1) - 1 for n, s in zip(lens, see)]))


def test_bad_parents_are_reported():
    """A parent that does not come before its child, and more tokens than the mask has bits; the other rows are right."""
    import w4a16_mixed_precision_gb300 as w4
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = w4.Kv4Batch(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), i(10), i(0, 5), 5, 5)
    ws = w4.Kv4Workspace(batch, 1, w4.Kv4Cache(1, 1, 64, 16))
    for parents, ref in (((-1, 0, 2, 1, 0), (1, 3, 4, 11, 17)), ((-1, 4, 0, 1, 1 << 30), (1, 2, 5, 10, 16)),
                         ((0, 0, -9, 2, 3), (1, 3, 4, 12, 28))):
        mask, positions = w4.kv4_tree(i(*parents), batch, ws)
        assert w4.device_status(ws) == 7 and w4.device_status(ws) == 0
        assert mask[:, 0].tolist() == list(ref)
        assert positions.tolist() == [4 + bin(x).count("1") for x in ref]
    many = w4.Kv4Batch(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), i(50), i(0, 40), 40, 32)
    mask, _ = w4.kv4_tree(torch.arange(-1, 39, dtype=torch.int32, device="cuda"), many, ws)
    assert w4.device_status(ws) == 7
    assert mask.shape == (40, 1) and mask[31:, 0].tolist() == [-1] * 9


TREES = [
    # lens, nq, hq, hkv, D, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([8], [8], 4, 2, 128, 16, 0),                          # nothing before the tree
    ([9, 30, 64, 70], [8, 3, 8, 8], 8, 2, 128, 16, 0),
    ([700], [8], 32, 32, 128, 64, 0),
    ([300, 65, 64], [1, 1, 1], 8, 8, 64, 32, 0),           # one token each
    ([513, 100, 33], [5, 2, 33], 3, 3, 64, 48, 0),
    ([2000, 77], [16, 13], 8, 2, 128, 128, 0),             # two groups of rows an instruction
    ([20000], [12], 8, 2, 128, 64, 0),                     # cut over many CTAs
    ([500, 40, 91], [6, 8, 5], 8, 2, 128, 16, 20),         # windows
    ([300, 100], [9, 40], 4, 4, 64, 16, 3),                # shorter than trees are deep
    ([64, 0, 20], [4, 0, 20], 4, 2, 128, 16, 0),
    ([i * 37 % 400 + 9 for i in range(60)], [1 + i % 8 for i in range(60)], 8, 2, 128, 32, 0),
    # many rows per key head
    ([65], [65], 1, 1, 64, 16, 0),
    ([100], [100], 4, 1, 128, 16, 0),
    ([1000, 200], [64, 64], 8, 1, 128, 64, 0),
    ([900], [25], 8, 1, 128, 64, 0),                       # one tile and a little
    ([777, 300], [61, 47], 7, 1, 64, 48, 0),
    ([5000], [60], 8, 2, 128, 16, 0),                      # few items: cut over CTAs
    ([3000, 2500], [40, 70], 16, 2, 64, 32, 1000),
    ([600], [130], 4, 2, 128, 32, 64),
    ([400, 90], [200, 90], 2, 1, 128, 64, 0),              # words of bits that blocks cut anywhere
    ([300] * 40, [70] * 40, 12, 6, 64, 64, 0),             # more items than SMs
    ([1500, 60, 30, 800], [40, 3, 30, 1], 8, 2, 128, 16, 0),   # both kernels
]


def setup(lens, nq, hq, hkv, D, page, seed, see):
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=seed)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q = np.random.default_rng(5).standard_normal((sum(nq), hq, D)).astype(np.float16)
    words = max(1, -(-max(nq) // 32))
    tree = cuda(np.concatenate([tree_ref.bits(s, words) for s in see]))
    return k, v, q, cache, batch, ws, tree


def near(y, ref, v, rows):
    """test_kv4_gpu.close, with the rounding of p s counted where the kernel for many rows served the request."""
    if rows <= 48 or not v.size:
        return close(y, ref, v)
    y = np.asarray(y, np.float64)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -12 * np.nanmax(np.abs(v)) + 2.0 ** -24
    tol = tol + 2.0 ** -11 * 8 / 15 * np.nanmax(np.nanmax(v, -1) - np.nanmin(v, -1))
    err = np.abs(y - ref)[~np.isnan(ref)]
    assert (err <= tol[~np.isnan(ref)]).all(), f"max error {err.max()}"


def check(y, q, k, v, lens, nq, see, D, window=0):
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
        near(yy, tree_ref.attention(qq, kv[b], vv[b], see[b], D ** -0.5, window), vv[b], nq[b] * q.shape[1] // k.shape[1])


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", TREES)
def test_tree_attention(lens, nq, hq, hkv, D, page, window):
    import w4a16_mixed_precision_gb300 as w4
    rng = np.random.default_rng(sum(lens) + hq)
    see = [tree_ref.sees(tree_ref.random_parents(n, rng)) for n in nq]
    k, v, q, cache, batch, ws, tree = setup(lens, nq, hq, hkv, D, page, sum(lens) + hq, see)
    y = w4.kv4_tree_attention(cuda(q), cache, batch, tree, ws, window=window)
    for _ in range(5):
        assert torch.equal(w4.kv4_tree_attention(cuda(q), cache, batch, tree, ws, window=window), y)
    assert w4.device_status(ws) == 0
    check(y, q, k, v, lens, nq, see, D, window)


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", [
    ([5000] + [70 + i for i in range(30)], [3] * 31, 24, 8, 64, 16, 0),        # a long cut one and many short
    ([70 + i for i in range(30)] + [5000], [2] * 31, 24, 8, 128, 32, 0),
    ([900 + 131 * i for i in range(24)], [5] * 24, 24, 8, 64, 16, 700),
    ([3000, 4, 5, 2000, 6, 900], [2, 4, 5, 1, 6, 3], 6, 3, 128, 64, 0),         # fewer blocks than warps
    ([65, 129, 700], [1, 1, 1], 2, 2, 64, 16, 0),
    ([10 + i * 61 % 2500 for i in range(100)], [1 + i % 4 for i in range(100)], 4, 2, 64, 48, 0),
])
def test_shares_that_begin_and_end_anywhere(lens, nq, hq, hkv, D, page, window):
    test_tree_attention(lens, nq, hq, hkv, D, page, window)


ANY = [([300, 40], [20, 40], 4, 2, 128, 16, 0), ([70, 66], [70, 66], 8, 1, 128, 64, 0), ([30, 5], [30, 5], 2, 2, 64, 32, 0),
       ([260], [100], 4, 1, 64, 16, 30), ([4000, 100], [33, 100], 8, 1, 64, 128, 0)]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", ANY)
def test_any_bits(lens, nq, hq, hkv, D, page, window):
    """Bits that are no tree: later tokens, not the row's own, none at all (zero where nothing comes before); bits
    behind the request's tokens are ignored, and so are more words than there are tokens."""
    import w4a16_mixed_precision_gb300 as w4
    rng = np.random.default_rng(sum(lens))
    see = []
    for n in nq:
        s = rng.random((n, n)) < 0.3
        s[0], s[-1], s[n // 2] = False, True, False
        see.append(s)
    k, v, q, cache, batch, ws, _ = setup(lens, nq, hq, hkv, D, page, sum(lens), see)
    words = -(-max(nq) // 32) + 2
    junk = [np.concatenate([s, rng.random((len(s), words * 32 - len(s))) < 0.5], 1) for s in see]
    tree = cuda(np.concatenate([tree_ref.bits(s, words) for s in junk]))
    y = w4.kv4_tree_attention(cuda(q), cache, batch, tree, ws, window=window)
    assert w4.device_status(ws) == 0
    check(y, q, k, v, lens, nq, see, D, window)
    t = 0
    for n, length, s in zip(nq, lens, see):
        for i in range(n):
            if length == n and not s[i].any():
                assert not y[t + i].any()
        t += n


@pytest.mark.parametrize("nq,hq", [(8, 4), (40, 8)])
def test_nan_stays_where_it_is_seen(nq, hq):
    """NaN and infinite keys and values of new tokens reach the rows that see them and no others."""
    import w4a16_mixed_precision_gb300 as w4
    lens, D, page = [150], 128, 16
    rng = np.random.default_rng(3)
    see = tree_ref.sees(tree_ref.random_parents(nq, rng))
    first = lens[0] - nq
    k, v, cache, batch, hist = make(lens, [nq], 1, D, page, seed=4)
    k[first + 3, 0, 5] = np.nan
    v[first + 5, 0, 7] = np.inf
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
    q = rng.standard_normal((nq, hq, D)).astype(np.float16)
    tree = cuda(tree_ref.bits(see, -(-nq // 32)))
    y = w4.kv4_tree_attention(cuda(q), cache, batch, tree, ws).cpu().numpy()
    assert w4.device_status(ws) == 0
    bad = see[:, 3] | see[:, 5]
    assert bad.any() and not bad.all()
    assert np.array_equal(np.isnan(y).any((1, 2)), bad) and np.array_equal(np.isnan(y).all((1, 2)), bad)
    ref = tree_ref.attention(q, kv_ref.values(k), kv_ref.values(v), see, D ** -0.5)
    near(y[~bad], ref[~bad], kv_ref.values(v)[:first + 3], nq * hq)


def test_a_run_of_tokens_is_causal_attention():
    import w4a16_mixed_precision_gb300 as w4
    for lens, nq, hq, hkv in (([900, 31], [6, 31], 4, 4), ([1200, 300], [100, 90], 8, 2)):
        see = [np.tril(np.ones((n, n), bool)) for n in nq]
        k, v, q, cache, batch, ws, tree = setup(lens, nq, hq, hkv, 128, 32, 7, see)
        dq = cuda(q)
        y, z = w4.kv4_tree_attention(dq, cache, batch, tree, ws), w4.kv4_attention(dq, cache, batch, ws)
        assert w4.device_status(ws) == 0
        top = float(np.abs(kv_ref.values(v)).max())
        assert float((y.double() - z.double()).abs().max()) <= 2 * (2.0 ** -11 + 2.0 ** -12) * top  # both within their tolerance
        check(y, q, k, v, lens, nq, see, 128)


def test_padded_rows_are_left_alone_and_graphs_replay():
    """Rows behind the last request stay as they were; a captured call replays on another stream, after the lengths
    and the tree changed in place, and two graphs share a workspace in turn."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [400, 90], [33, 20], 8, 1, 64, 16
    rng = np.random.default_rng(8)
    see = [tree_ref.sees(tree_ref.random_parents(n, rng)) for n in nq]
    k, v, q, cache, batch, ws, tree = setup(lens, nq, hq, hkv, D, page, 9, see)
    pad = 11
    T = sum(nq) + pad
    ws = w4.Kv4Workspace(w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, T, max(nq)), hq, cache)
    qp = torch.full((T, hq, D), float("nan"), dtype=torch.float16, device="cuda")
    qp[:-pad] = cuda(q)
    tp = torch.full((T, tree.shape[1]), -1, dtype=torch.int32, device="cuda")
    tp[:-pad] = tree
    padded = w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, T, max(nq))
    out = torch.full((T, hq, D), 7.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        w4.kv4_tree_attention_into(qp, cache, padded, tp, ws, out)
    s.synchronize()
    assert (out[-pad:] == 7).all()
    check(out[:-pad], q, k, v, lens, nq, see, D)
    graphs, outs = [], []
    for _ in range(2):
        outs.append(torch.zeros_like(out))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            w4.kv4_tree_attention_into(qp, cache, padded, tp, ws, outs[-1])
    see = [tree_ref.sees(tree_ref.random_parents(n, rng)) for n in nq]
    tp[:-pad] = cuda(np.concatenate([tree_ref.bits(x, tree.shape[1]) for x in see]))
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert w4.device_status(ws) == 0
    for o in outs:
        check(o[:-pad], q, k, v, lens, nq, see, D)
        assert not o[-pad:].any()


def test_one_workspace_for_trees_and_runs_in_turn():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [3000, 40], [60, 2], 8, 1, 128, 64
    rng = np.random.default_rng(10)
    see = [tree_ref.sees(tree_ref.random_parents(n, rng)) for n in nq]
    k, v, q, cache, batch, ws, tree = setup(lens, nq, hq, hkv, D, page, 11, see)
    dq = cuda(q)
    y, z = w4.kv4_tree_attention(dq, cache, batch, tree, ws), w4.kv4_attention(dq, cache, batch, ws)
    few = w4.Kv4Batch(batch.page_table, batch.lengths, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), 2, 1)
    for _ in range(3):
        assert torch.equal(w4.kv4_attention(dq, cache, batch, ws), z)
        w4.kv4_tree_attention(dq[:2], cache, few, torch.ones((2, 1), dtype=torch.int32, device="cuda"), ws)
        assert torch.equal(w4.kv4_tree_attention(dq, cache, batch, tree, ws), y)
    assert w4.device_status(ws) == 0
    check(y, q, k, v, lens, nq, see, D)


@pytest.mark.parametrize("nq", [7, 70])
def test_bad_entries_are_reported_and_not_followed(nq):
    import w4a16_mixed_precision_gb300 as w4
    lens, hq, hkv, D, page = [90, 160], 4, 2, 128, 16
    rng = np.random.default_rng(12)
    see = [tree_ref.sees(tree_ref.random_parents(nq, rng)) for _ in lens]
    k, v, q, cache, batch, ws, tree = setup(lens, [nq, nq], hq, hkv, D, page, 13, see)
    dq = cuda(q)
    ref = tree_ref.attention(q[:nq], kv_ref.values(k)[:90], kv_ref.values(v)[:90], see[0], D ** -0.5)
    for change in ("page", "negative page", "length", "short", "start", "words"):
        table, length, start, bits = batch.page_table.clone(), batch.lengths.clone(), batch.q_start.clone(), tree
        if change == "page":
            table[1, 2] = cache.n_pages
        elif change == "negative page":
            table[1, 0] = -7
        elif change == "length":
            length[1] = table.shape[1] * page + 1
        elif change == "short":
            length[1] = 5
        elif change == "start":
            start[2] = 2 * nq + 1
        else:
            if nq <= 32:
                continue
            bits = tree[:, :1].contiguous()
        y = w4.kv4_tree_attention(dq, cache, w4.Kv4Batch(table, length, start, 2 * nq, nq), bits, ws)
        assert w4.device_status(ws) == 7, change
        if change != "words":
            near(y[:nq].cpu().numpy(), ref, kv_ref.values(v), nq * 2)
    y = w4.kv4_tree_attention(dq, cache, batch, tree, ws)
    assert w4.device_status(ws) == 0
    near(y[:nq].cpu().numpy(), ref, kv_ref.values(v), nq * 2)


def test_refusals():
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make([40], [2], 2, 128, 16, seed=14)
    ws = w4.Kv4Workspace(batch, 4, cache)
    q = torch.zeros((2, 4, 128), dtype=torch.float16, device="cuda")
    tree = torch.ones((2, 1), dtype=torch.int32, device="cuda")
    for bad in (tree.long(), tree.cpu(), tree[:1], tree[:, 0], tree.expand(2, 3), tree.bool()):
        with pytest.raises(ValueError):
            w4.kv4_tree_attention(q, cache, batch, bad, ws)
    for bad in (q.float(), q.cpu(), q[:1], q[:, :, :64]):
        with pytest.raises(ValueError):
            w4.kv4_tree_attention(bad, cache, batch, tree, ws)
    for args in (dict(window=-1), dict(scale=float("inf"))):
        with pytest.raises(w4.MarlinError):
            w4.kv4_tree_attention(q, cache, batch, tree, ws, **args)
    with pytest.raises(w4.MarlinError):
        w4.kv4_tree_attention(q, cache, batch, tree[:, :0], ws)
    parents = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    for bad in (parents.long(), parents.cpu(), parents[:1], parents[:, None]):
        with pytest.raises(ValueError):
            w4.kv4_tree(bad, batch, ws)
    none = w4.Kv4Batch(batch.page_table, batch.lengths, torch.zeros_like(batch.q_start), 0, 0)
    assert w4.kv4_tree_attention(q[:0], cache, none, tree[:0], ws).shape == (0, 4, 128)
    assert [t.shape[0] for t in w4.kv4_tree(parents[:0], none, ws)] == [0, 0]
    assert w4.device_status(ws) == 0
