"""The operators for drafted trees in a row, as a server uses them: masks and positions, rotary and append, attention,
the kept tokens' entries moved together in two layers' caches, single tokens after them, a fork that shares pages and
copies the last one.  Every attention output against 64 bits, over the tokens that a request has kept.

Tolerances are those of test_kv4_tree_gpu.py, derived there.  The keys of the reference are rotated in fp32 and rounded to
fp16 like the operator's (bit for bit: test_kv4_rope_gpu.py)."""
import os
import sys

import numpy as np
import pytest

import kv_ref
import tree_ref
from test_kv4_gpu import _built  # noqa: F401
from test_kv4_tree_gpu import near

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return cuda(np.asarray(x, np.int32))


class Request:
    def __init__(self, layers, hkv, D):
        self.pages = []
        self.k = [np.zeros((0, hkv, D), np.float16) for _ in range(layers)]  # rotated keys of the kept tokens
        self.v = [np.zeros((0, hkv, D), np.float16) for _ in range(layers)]

    @property
    def length(self):
        return len(self.k[0])


@pytest.mark.parametrize("hq,hkv,D,page,sizes", [(4, 2, 64, 16, (9, 30, 3)), (16, 2, 128, 32, (40, 13, 64)), (8, 8, 128, 48, (5, 8, 1))])
def test_verify_keep_and_fork(hq, hkv, D, page, sizes):
    import w4a16_mixed_precision_gb300 as w4
    layers, n_pages, max_pages = 2, 60, 14
    rng = np.random.default_rng(hq * D)
    caches = [w4.Kv4Cache(n_pages, hkv, D, page) for _ in range(layers)]
    for c in caches:
        c.buf.random_(0, 256)
    pool = w4.Kv4Pages(n_pages, page)
    rope = w4.Kv4Rope.from_theta(D, 2000)
    cos, sin = (t.cpu().numpy() for t in rope.table.unbind(-1))
    pairs = [0] * (D // 2)
    ws = w4.Kv4Workspace(w4.Kv4Batch(i32([[0]]), i32([0]), i32([0, 400]), 400, 400), hq, caches[0])
    requests = [Request(layers, hkv, D) for _ in sizes]

    def batch(new):
        table = np.full((len(requests), max_pages), -1, np.int32)
        for b, (r, n) in enumerate(zip(requests, new)):
            r.pages += pool.take(max(0, -(-(r.length + n) // page) - len(r.pages)))
            table[b, :len(r.pages)] = r.pages
        return w4.Kv4Batch(cuda(table), i32([r.length + n for r, n in zip(requests, new)]),
                           i32(np.concatenate([[0], np.cumsum(new)])), sum(new), max(new))

    def step(trees, keep, causal=False):
        """trees: each request's parents; keep: what it keeps of them."""
        new = [len(t) for t in trees]
        now = batch(new)
        mask, positions = w4.kv4_tree(i32(np.concatenate(trees)), now, ws)
        see = [tree_ref.sees(t) for t in trees]
        at = np.concatenate([r.length + s.sum(1) - 1 for r, s in zip(requests, see)])
        assert np.array_equal(positions.cpu().numpy(), at)
        after = []
        for layer, cache in enumerate(caches):
            qkv = rng.standard_normal((sum(new), hq + 2 * hkv, D)).astype(np.float16)
            q, k, v = cuda(qkv).split([hq, hkv, hkv], dim=1)
            q = w4.kv4_rope_append(q, k, v, positions, rope, cache, now, ws)
            y = w4.kv4_attention(q, cache, now, ws) if causal else w4.kv4_tree_attention(q, cache, now, mask, ws)
            qr, kr = (tree_ref.rotate(x, at[None], cos, sin, pairs, False)[0] for x in (qkv[:, :hq], qkv[:, hq:hq + hkv]))
            t, rows = 0, []
            for r, s, n in zip(requests, see, new):
                kk, vv = np.concatenate([r.k[layer], kr[t:t + n]]), np.concatenate([r.v[layer], qkv[t:t + n, hq + hkv:]])
                ref = tree_ref.attention(qr[t:t + n], kv_ref.values(kk), kv_ref.values(vv), s, D ** -0.5)
                near(y[t:t + n].cpu().numpy(), ref, kv_ref.values(vv), n * hq // hkv)
                rows.append((kr[t:t + n], qkv[t:t + n, hq + hkv:]))
                t += n
            after.append(rows)
        index = np.concatenate([np.concatenate([x, np.zeros(n - len(x))]) for x, n in zip(keep, new)])
        lengths = w4.kv4_compact(caches, now, i32(index), i32([len(x) for x in keep]), ws)
        for layer, rows in enumerate(after):
            for r, x, (kr, vr) in zip(requests, keep, rows):
                r.k[layer], r.v[layer] = np.concatenate([r.k[layer], kr[x]]), np.concatenate([r.v[layer], vr[x]])
        assert lengths.tolist() == [r.length for r in requests]
        for r in requests:
            spare = -(-r.length // page)
            pool.free(r.pages[spare:])
            del r.pages[spare:]
        assert w4.device_status(ws) == 0

    def path(parents):
        """From a random token up to the root."""
        at, out = int(rng.integers(len(parents))), []
        while at >= 0:
            out.append(at)
            at = int(parents[at])
        return np.array(out[::-1])

    # prompts: runs of tokens, all kept; one request has none
    prompts = [np.arange(-1, n - 1, dtype=np.int32) for n in (50, 17, 0)]
    step(prompts, [np.arange(len(p)) for p in prompts], causal=True)
    for _ in range(2):
        trees = [tree_ref.random_parents(n, rng) for n in sizes]
        step(trees, [path(t) for t in trees])
    # the first request forks: both go on, each on its own
    one = Request(layers, hkv, D)
    one.pages, copies = pool.fork(requests[0].pages, requests[0].length)
    one.k, one.v = [x.copy() for x in requests[0].k], [x.copy() for x in requests[0].v]
    assert len(copies) == (requests[0].length % page > 0) and all(pool.shared(p) for p in one.pages[:requests[0].length // page])
    w4.kv4_copy_pages(caches, i32([a for a, _ in copies]), i32([b for _, b in copies]), ws)
    requests.append(one)
    for _ in range(2):
        trees = [tree_ref.random_parents(n, rng) for n in (*sizes, 20)]
        step(trees, [path(t) for t in trees])
    # one request leaves, the others have single tokens
    pool.free(requests.pop(0).pages)
    single = [np.array([-1], np.int32)] * 3
    step(single, [np.array([0])] * 3, causal=True)
    step(single, [np.array([0])] * 3)
    for r in requests:
        pool.free(r.pages)
    assert pool.free_pages == n_pages


def test_the_example_runs():
    """More than a token a request and step, and every page is free or held."""
    import verify_trees
    server, got = verify_trees.serve(requests=3, steps=9, layers=2, hidden=512, heads=4, kv_heads=2, draft=9)
    assert len(got) == 9 and [len(x) for x in got] == [3] * 3 + [4] * 6
    assert all(n >= 1 for x in got for n in x)
    for r, n in zip(server.requests, [sum(x[b] for x in got if len(x) > b) for b in range(4)]):
        assert r.length == len(r.tokens) - 1 and len(r.pages) == -(-r.length // 16)
    held = {p for r in server.requests for p in r.pages}
    assert server.pages.free_pages + len(held) == 64 * 4
