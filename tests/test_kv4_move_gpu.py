"""Moving what the caches hold, on the GPU: kept tokens read back as what was appended for them, bit for bit, every
other byte of the caches stays as it was; pages are copied byte for byte.
"""
import numpy as np
import pytest

import kv_ref
from test_kv4_gpu import _built, make  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return cuda(np.asarray(x, np.int32))


def starts(n):
    return i32(np.concatenate([[0], np.cumsum(n)]))


def filled(lens, nq, hkv, D, page, layers, seed):
    """Caches of several layers with the requests' whole histories in them; pages beyond them are free."""
    import w4a16_mixed_precision_gb300 as w4
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    n_pages = 2 * sum(per) + 2
    order = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((2, len(lens), max(max(per), 1)), -1, np.int32)
    at = 0
    for i in range(2):
        for b, n in enumerate(per):
            tables[i, b, :n] = order[at:at + n]
            at += n
    caches = [w4.Kv4Cache(n_pages, hkv, D, page) for _ in range(layers)]
    H = sum(lens)
    hist = w4.Kv4Batch(i32(tables[0]), i32(lens), starts(lens), H, max(lens))
    batch = w4.Kv4Batch(i32(tables[0]), i32(lens), starts(nq), sum(nq), max(nq))
    ws = w4.Kv4Workspace(batch, hkv, caches[0])
    kv = []
    for cache in caches:
        cache.buf.random_(0, 256)
        k, v = (rng.standard_normal((H, hkv, D)).astype(np.float16) for _ in "kv")
        w4.kv4_append(cuda(k), cuda(v), cache, hist, ws)
        kv.append((kv_ref.values(k).astype(np.float16), kv_ref.values(v).astype(np.float16)))
    return caches, batch, ws, kv, i32(tables[1])


def read(cache, table, lens, ws):
    import w4a16_mixed_precision_gb300 as w4
    k, v = w4.kv4_read(cache, w4.Kv4Batch(table, i32(lens), starts(lens), sum(lens), max(lens)), ws)
    return k.cpu().numpy(), v.cpu().numpy()


def padded(index, nq):
    return i32(np.concatenate([np.concatenate([x, np.full(n - len(x), -99)]) for x, n in zip(index, nq)]))


def check(caches, table, ws, kv, lens, nq, index, new):
    """The requests' histories with the kept tokens in place of the new ones."""
    at, want = 0, []
    for n, length, x in zip(nq, lens, index):
        want += list(range(at, at + length - n)) + [at + length - n + i for i in x]
        at += length
    for cache, (k, v) in zip(caches, kv):
        got = read(cache, table, new, ws)
        assert np.array_equal(got[0], k[want]) and np.array_equal(got[1], v[want])


KEEP = [
    # lens, nq, hkv, D, page, layers
    ([1], [1], 1, 64, 16, 1),
    ([9, 30, 100], [8, 3, 61], 2, 128, 16, 3),
    ([40, 17, 16, 33], [16, 16, 16, 16], 8, 64, 48, 2),
    ([130, 0, 77], [64, 0, 77], 3, 128, 32, 1),
    ([700, 300], [400, 300], 2, 64, 64, 2),         # several rounds of a warp
    ([3000], [2900], 1, 128, 128, 1),
    ([64] * 50, [5] * 50, 4, 128, 16, 2),
]


@pytest.mark.parametrize("lens,nq,hkv,D,page,layers", KEEP)
@pytest.mark.parametrize("share", [0.1, 0.6, 1.0])
def test_keeps_tokens_in_their_pages(lens, nq, hkv, D, page, layers, share):
    import w4a16_mixed_precision_gb300 as w4
    caches, batch, ws, kv, _ = filled(lens, nq, hkv, D, page, layers, seed=sum(lens))
    rng = np.random.default_rng(sum(nq))
    index = [np.flatnonzero(rng.random(n) < share) for n in nq]
    before = [c.buf.clone() for c in caches]
    new = w4.kv4_compact(caches if layers > 1 else caches[0], batch, padded(index, nq), i32([len(x) for x in index]), ws)
    assert w4.device_status(ws) == 0
    assert new.tolist() == [length - n + len(x) for length, n, x in zip(lens, nq, index)]
    check(caches, batch.page_table, ws, kv, lens, nq, index, new.tolist())
    # and what was not kept is where it was: all positions behind the kept ones read as before
    for cache, old, (k, v) in zip(caches, before, kv):
        got = read(cache, batch.page_table, lens, ws)
        at = 0
        for n, length, x in zip(nq, lens, index):
            a, b = at + length - n + len(x), at + length
            assert np.array_equal(got[0][a:b], k[a:b]) and np.array_equal(got[1][a:b], v[a:b])
            at = b


@pytest.mark.parametrize("lens,nq,hkv,D,page,layers", KEEP)
def test_gathers_tokens_into_other_pages(lens, nq, hkv, D, page, layers):
    """In any order, tokens several times or not at all; the old pages keep what they held."""
    import w4a16_mixed_precision_gb300 as w4
    caches, batch, ws, kv, into = filled(lens, nq, hkv, D, page, layers, seed=sum(lens) + 1)
    rng = np.random.default_rng(sum(nq))
    index = [rng.integers(0, n, rng.integers(0, n + 1)) if n else np.zeros(0, int) for n in nq]
    before = [read(c, batch.page_table, lens, ws) for c in caches]
    new = w4.kv4_compact(caches, batch, padded(index, nq), i32([len(x) for x in index]), ws, into=into)
    assert w4.device_status(ws) == 0
    assert new.tolist() == [length - n + len(x) for length, n, x in zip(lens, nq, index)]
    # read the kept tokens alone: those before them are not in the new pages
    count = [len(x) for x in index]
    tokens = w4.Kv4Batch(into, new, starts(count), sum(count), max(count))
    at, want = 0, []
    for n, length, x in zip(nq, lens, index):
        want += [at + length - n + i for i in x]
        at += length
    for cache, (k, v), old in zip(caches, kv, before):
        if want:
            got = w4.kv4_read(cache, tokens, ws)
            assert np.array_equal(got[0].cpu().numpy(), k[want]) and np.array_equal(got[1].cpu().numpy(), v[want])
        now = read(cache, batch.page_table, lens, ws)
        assert np.array_equal(now[0], old[0], equal_nan=True) and np.array_equal(now[1], old[1], equal_nan=True)
    assert w4.device_status(ws) == 0


@pytest.mark.parametrize("lens,nq,hkv,D,page,layers", [
    ([1990, 27, 1201, 0, 64], [1985, 7, 1200, 0, 64], 5, 64, 16, 7),   # 4 of 35 heads together, across the caches' ends
    ([4000, 133, 1600], [4000, 33, 1590], 3, 128, 64, 17),             # 7 of 51
    ([300] * 50, [290] * 50, 4, 128, 48, 5),                           # 4 of 20
])
def test_gathers_several_heads_together(lens, nq, hkv, D, page, layers):
    """With so much to move that a warp takes several heads (on 152 SMs as many as said)."""
    test_gathers_tokens_into_other_pages(lens, nq, hkv, D, page, layers)


def test_bytes_that_are_not_named_stay():
    """In a cache of random bytes nothing but the kept positions' entries changes."""
    import w4a16_mixed_precision_gb300 as w4
    hkv, D, page = 2, 128, 32
    for into in (False, True):
        caches, batch, ws, _, other = filled([70, 45], [40, 30], hkv, D, page, 1, seed=5)
        cache = caches[0]
        cache.buf.random_(0, 256)
        index = [np.array([0, 3, 4, 17, 39]), np.array([1, 2, 29])]
        before = cache.buf.clone()
        w4.kv4_compact(cache, batch, padded(index, [40, 30]), i32([5, 3]), ws, into=other if into else None)
        assert w4.device_status(ws) == 0
        # which bytes a position has: those that an append of it writes
        table = other if into else batch.page_table
        touched = torch.zeros_like(cache.buf, dtype=torch.bool)
        for fill in (0, 255):
            probe = w4.Kv4Cache(cache.n_pages, hkv, D, page)
            probe.buf.fill_(fill)
            x = torch.full((8, hkv, D), 1.5, dtype=torch.float16, device="cuda")
            x[..., ::2] = -3.25
            w4.kv4_append(x, x, probe, w4.Kv4Batch(table, i32([35, 18]), i32([0, 5, 8]), 8, 5), ws)
            touched |= probe.buf != fill
        assert torch.equal(cache.buf[~touched], before[~touched])
        assert int(touched.sum()) == 8 * hkv * (D + 8)


def test_requests_that_do_not_fit_are_left_alone():
    """Indexes that do not ascend or lie outside, counts outside, bad starts and pages: reported, the request as it was,
    the others moved."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hkv, D, page = [50, 90], [20, 60], 2, 64, 16
    for change in ("equal", "descending", "high", "negative", "count", "negative count", "start", "length"):
        caches, batch, ws, kv, _ = filled(lens, nq, hkv, D, page, 2, seed=6)
        index = np.zeros(80, np.int32)
        index[:3], index[20:24] = (0, 5, 9), (1, 7, 30, 59)
        kept, start, length = [3, 4], batch.q_start.clone(), batch.lengths.clone()
        if change == "equal":
            index[21] = 1
        elif change == "descending":
            index[22] = 3
        elif change == "high":
            index[23] = 60
        elif change == "negative":
            index[20] = -1
        elif change == "count":
            kept[1] = 61
        elif change == "negative count":
            kept[1] = -1
        elif change == "start":
            start[2] = 81
        else:
            length[1] = 59
        before = [read(c, batch.page_table, lens, ws) for c in caches]
        new = w4.kv4_compact(caches, w4.Kv4Batch(batch.page_table, length, start, 80, 60), i32(index), i32(kept), ws)
        assert w4.device_status(ws) == 7, change
        assert new.tolist() == [33, int(length[1])], change
        for cache, old, (k, v) in zip(caches, before, kv):
            got = read(cache, batch.page_table, lens, ws)
            assert np.array_equal(got[0][50:], old[0][50:]) and np.array_equal(got[1][50:], old[1][50:])
            assert np.array_equal(got[0][30:33], k[[30, 35, 39]]) and np.array_equal(got[1][30:33], v[[30, 35, 39]])


def test_bad_pages_are_not_followed():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hkv, D, page = [100], [90], 2, 128, 16
    for into in (False, True):
        caches, batch, ws, kv, other = filled(lens, nq, hkv, D, page, 1, seed=7)
        table = (other if into else batch.page_table).clone()
        table[0, 2] = caches[0].n_pages
        index = np.arange(90, dtype=np.int32)
        args = dict(into=table) if into else {}
        src = batch if into else w4.Kv4Batch(table, batch.lengths, batch.q_start, 90, 90)
        w4.kv4_compact(caches, src, i32(index), i32([90]), ws, **args)
        assert w4.device_status(ws) == 7
        if into:   # a table of fewer pages than the kept tokens need
            w4.kv4_compact(caches, batch, i32(index), i32([90]), ws, into=other[:, :3].contiguous())
            assert w4.device_status(ws) == 7
        assert w4.device_status(ws) == 0


def test_no_tokens_and_none_kept():
    import w4a16_mixed_precision_gb300 as w4
    caches, batch, ws, kv, into = filled([30, 20], [5, 20], 2, 64, 16, 2, seed=8)
    before = [c.buf.clone() for c in caches]
    assert w4.kv4_compact(caches, batch, i32([0] * 25), i32([0, 0]), ws).tolist() == [25, 0]
    assert w4.kv4_compact(caches, batch, i32([0] * 25), i32([0, 0]), ws, into=into).tolist() == [25, 0]
    none = w4.Kv4Batch(batch.page_table, batch.lengths, torch.zeros_like(batch.q_start), 0, 0)
    assert w4.kv4_compact(caches, none, i32([]), i32([0, 0]), ws).tolist() == [30, 20]
    w4.kv4_copy_pages(caches, i32([]), i32([]), ws)
    w4.kv4_copy_pages(caches, i32([-1, -7]), i32([0, 1]), ws)
    assert w4.device_status(ws) == 0
    assert all(torch.equal(c.buf, b) for c, b in zip(caches, before))


@pytest.mark.parametrize("n_pages,hkv,D,page,layers,pairs", [(4, 1, 64, 16, 1, 1), (60, 3, 128, 48, 5, 29), (9, 8, 128, 256, 2, 4),
                                                             (30, 2, 64, 16, 131, 15)])
def test_copies_pages(n_pages, hkv, D, page, layers, pairs):
    import w4a16_mixed_precision_gb300 as w4
    caches = [w4.Kv4Cache(n_pages, hkv, D, page) for _ in range(layers)]
    ws = w4.Kv4Workspace(w4.Kv4Batch(i32([[0]]), i32([0]), i32([0, 0]), 0, 0), hkv, caches[0])
    order = np.random.default_rng(n_pages).permutation(n_pages)
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs]
    src[pairs // 2:pairs // 2 + 2] = src[0]     # one page for several
    skip = pairs - 1 if pairs > 4 else None
    if skip:
        src[skip] = -1
    want = []
    for c in caches:
        c.buf.random_(0, 256)
        pages = c.buf.clone().view(n_pages, -1)
        for a, b in zip(src, dst):
            if a >= 0:
                pages[b] = pages[a]
        want.append(pages.view(-1))
    w4.kv4_copy_pages(caches, i32(src), i32(dst), ws)
    assert w4.device_status(ws) == 0
    assert all(torch.equal(c.buf, x) for c, x in zip(caches, want))
    for a, b in ((n_pages, 0), (0, n_pages), (0, -1), (1 << 30, 1)):
        w4.kv4_copy_pages(caches, i32([a]), i32([b]), ws)
        assert w4.device_status(ws) == 7
    assert all(torch.equal(c.buf, x) for c, x in zip(caches, want))


def test_pages_beyond_32_bits():
    """A cache of more than 4 GiB: its last pages are copied and compacted."""
    import w4a16_mixed_precision_gb300 as w4
    hkv, D, page = 8, 128, 1024
    n_pages = (5 << 30) // (hkv * page * (D + 8)) + 1
    cache = w4.Kv4Cache(n_pages, hkv, D, page)
    last = i32([[n_pages - 1]])
    batch = w4.Kv4Batch(last, i32([40]), i32([0, 40]), 40, 40)
    ws = w4.Kv4Workspace(batch, hkv, cache)
    rng = np.random.default_rng(12)
    k, v = (rng.standard_normal((40, hkv, D)).astype(np.float16) for _ in "kv")
    w4.kv4_append(cuda(k), cuda(v), cache, batch, ws)
    w4.kv4_copy_pages(cache, i32([n_pages - 1]), i32([n_pages - 2]), ws)
    index = i32(np.concatenate([[3, 11, 30, 39], np.zeros(36)]))
    w4.kv4_compact(cache, w4.Kv4Batch(i32([[n_pages - 2]]), batch.lengths, batch.q_start, 40, 40), index, i32([4]), ws)
    w4.kv4_compact(cache, batch, index, i32([4]), ws, into=i32([[n_pages - 3]]))
    assert w4.device_status(ws) == 0
    for page_ in (n_pages - 2, n_pages - 3):
        got = read(cache, i32([[page_]]), [4], ws)
        for x, y in zip(got, (k, v)):
            assert np.array_equal(x, kv_ref.values(y)[[3, 11, 30, 39]].astype(np.float16))
    assert int(cache.buf[:1 << 20].max()) == 0


def test_more_caches_than_one_launch_takes():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, index = [9, 5], [6, 5], [np.array([1, 4]), np.array([0, 2, 3, 4])]
    for other in (False, True):
        caches, batch, ws, kv, into = filled(lens, nq, 1, 64, 16, 130, seed=11)
        new = w4.kv4_compact(caches, batch, padded(index, nq), i32([2, 4]), ws, into=into if other else None)
        assert w4.device_status(ws) == 0 and new.tolist() == [5, 4]
        if not other:
            check(caches, batch.page_table, ws, kv, lens, nq, index, [5, 4])
        else:
            for cache, (k, v) in zip(caches, kv):
                got = w4.kv4_read(cache, w4.Kv4Batch(into, new, starts([2, 4]), 6, 4), ws)
                assert np.array_equal(got[0].cpu().numpy(), k[[4, 7, 9, 11, 12, 13]])
                assert np.array_equal(got[1].cpu().numpy(), v[[4, 7, 9, 11, 12, 13]])


def test_on_another_stream_and_in_a_graph():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq = [60, 45], [30, 17]
    caches, batch, ws, kv, _ = filled(lens, nq, 2, 128, 16, 2, seed=9)
    index, kept = i32(np.zeros(47)), i32([0, 0])
    first = i32([[0], [1]])
    src, dst = first[:, 0].clone(), i32([caches[0].n_pages - 1, caches[0].n_pages - 2])
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lengths = w4.kv4_compact(caches, batch, index, kept, ws)
        w4.kv4_copy_pages(caches, src, dst, ws)
    which = [np.array([2, 20]), np.array([0, 1, 16])]
    index.copy_(padded(which, nq))
    kept.copy_(i32([2, 3]))
    src.fill_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert w4.device_status(ws) == 0 and lengths.tolist() == [32, 31]
    check(caches, batch.page_table, ws, kv, lens, nq, which, [32, 31])


def test_refusals():
    import w4a16_mixed_precision_gb300 as w4
    caches, batch, ws, _, into = filled([30], [4], 2, 64, 16, 2, seed=10)
    index, kept = i32([0, 1, 2, 3]), i32([2])
    other = w4.Kv4Cache(caches[0].n_pages, 2, 64, 32)
    for bad in (dict(index=index.long()), dict(index=index[:3]), dict(kept=i32([1, 1])), dict(kept=kept.cpu()), dict(caches=[]),
                dict(caches=[caches[0], other]), dict(into=into[0]), dict(into=into.long())):
        args = dict(dict(caches=caches, index=index, kept=kept, into=None), **bad)
        with pytest.raises(ValueError):
            w4.kv4_compact(args["caches"], batch, args["index"], args["kept"], ws, into=args["into"])
    for call in (lambda c: w4.kv4_compact(c, batch, index, kept, ws), lambda c: w4.kv4_copy_pages(c, i32([0]), i32([1]), ws)):
        with pytest.raises(w4.MarlinError) as e:
            call([caches[0], caches[1], caches[0]])   # one of them twice
        assert e.value.status == 1
    for s, d in ((i32([0, 1]), i32([2])), (i32([[0]]), i32([[1]])), (i32([0]).long(), i32([1])), (i32([0]).cpu(), i32([1]))):
        with pytest.raises(ValueError):
            w4.kv4_copy_pages(caches, s, d, ws)
    assert w4.device_status(ws) == 0
