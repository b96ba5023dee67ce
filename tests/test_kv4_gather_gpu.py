"""Kept tokens into other pages where a request's indexes or counts do not fit: reported, nothing of the request moved,
its length as it was, the others moved.  Every byte of the caches is compared with a call in which the request keeps
nothing."""
import numpy as np
import pytest

from test_kv4_gpu import _built  # noqa: F401
from test_kv4_move_gpu import filled, i32

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SIZES = [
    # lens, nq, hkv, D, page, layers
    ([50, 90, 70], [20, 60, 31], 2, 64, 16, 2),            # a warp has a request's tokens
    ([5, 9, 8], [5, 9, 8], 1, 128, 16, 130),               # more caches than a launch takes
    ([900, 5100, 2600], [880, 5000, 2600], 3, 128, 48, 5),
    ([3000, 40000, 2000], [3000, 39000, 1], 4, 64, 64, 2),  # several heads a warp
]


@pytest.mark.parametrize("lens,nq,hkv,D,page,layers", SIZES)
@pytest.mark.parametrize("claimed", [None, 1])
def test_a_request_that_does_not_fit_is_left_alone(lens, nq, hkv, D, page, layers, claimed):
    import w4a16_mixed_precision_gb300 as w4
    caches, batch, ws, kv, into = filled(lens, nq, hkv, D, page, layers, seed=sum(lens))
    rng = np.random.default_rng(sum(nq))
    T, start = sum(nq), np.concatenate([[0], np.cumsum(nq)])
    batch = w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, T, claimed or max(nq))  # max_q is a hint
    index = np.concatenate([rng.integers(0, n, n) for n in nq])
    kept = np.array([nq[0], nq[1] - 2, nq[2] // 2])
    index[start[1] + kept[1]:start[2]] = (-5, 1 << 30)          # behind the kept ones: not looked at
    before = [c.buf.clone() for c in caches]
    want = None
    bad = [("low", 0), ("high", 0), ("high", nq[1] // 3), ("low", nq[1] // 2), ("high", int(kept[1]) - 1), ("far", 5 % kept[1]),
           ("count", 0), ("negative count", 0), ("length", 0), ("start", 0)]
    for change, at in bad:
        x, n, length, starts = index.copy(), kept.copy(), batch.lengths.clone(), batch.q_start.clone()
        if change in ("low", "high", "far"):
            x[start[1] + at] = {"low": -1, "high": nq[1], "far": -(1 << 31)}[change]
        elif change == "count":
            n[1] = nq[1] + 1
        elif change == "negative count":
            n[1] = -1
        elif change == "length":
            length[1] = nq[1] - 1
        else:
            starts[2] = start[1] - 1                            # the third begins before the second's first, too
        for c, b in zip(caches, before):
            c.buf.copy_(b)
        new = w4.kv4_compact(caches, w4.Kv4Batch(batch.page_table, length, starts, T, batch.max_q), i32(x), i32(n), ws, into=into)
        if change == "start":
            assert w4.device_status(ws) == 7
            assert new[:2].tolist() == [lens[0] - nq[0] + kept[0], lens[1]]
            continue
        got = [c.buf.clone() for c in caches]
        # what was reported is not read yet: a call without a fault is right all the same
        for c, b in zip(caches, before):
            c.buf.copy_(b)
        n[1] = 0
        good = w4.kv4_compact(caches, batch, i32(index), i32(n), ws, into=into)
        assert w4.device_status(ws) == 7 and w4.device_status(ws) == 0, change
        ends = [a - b + c for a, b, c in zip(lens, nq, kept)]
        assert new.tolist() == [ends[0], int(length[1]), ends[2]], (change, at)
        assert good.tolist() == [ends[0], lens[1] - nq[1], ends[2]]
        assert all(torch.equal(a, c.buf) for a, c in zip(got, caches)), (change, at)
        if want is None:
            want = got
            assert not any(torch.equal(a, b) for a, b in zip(want, before))
        assert all(torch.equal(a, b) for a, b in zip(want, got)), (change, at)


def test_in_a_graph():
    """The indexes change in place between replays: to bad ones and back."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq = [3000, 800], [2900, 800]
    caches, batch, ws, kv, into = filled(lens, nq, 2, 128, 16, 3, seed=3)
    rng = np.random.default_rng(3)
    one = np.concatenate([rng.integers(0, n, n) for n in nq])
    index, kept = i32(one), i32([1500, 700])
    w4.kv4_compact(caches, batch, index, kept, ws, into=into)    # loaded before the capture
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        new = w4.kv4_compact(caches, batch, index, kept, ws, into=into)
    for c in caches:
        c.buf.zero_()
        # (what the pages hold does not matter here, only whether it is moved)
        c.buf.view(-1)[:].random_(0, 256)
    for bad in (True, False, True):
        x = one.copy()
        if bad:
            x[77] = 2900
        index.copy_(i32(x))
        before = [c.buf.clone() for c in caches]
        g.replay()
        torch.cuda.synchronize()
        assert w4.device_status(ws) == (7 if bad else 0)
        assert new.tolist() == [3000 if bad else 1600, 700]
        first = into[0, :-(-1600 // 16)].long()
        for c, b in zip(caches, before):
            pages, old = c.buf.view(c.n_pages, -1), b.view(c.n_pages, -1)
            assert torch.equal(pages[first], old[first]) == bad
