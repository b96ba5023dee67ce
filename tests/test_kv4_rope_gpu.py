"""Rotary positions with the append, on the GPU: the rotated queries are, bit for bit, fp32 products and sums rounded
one by one and then to fp16, and the cache holds what kv4_append makes of the keys rotated so.  Against 64 bits the
rotated channels are off by the fp16 rounding and three fp32 ones of |x1| + |x2| (the entries are at most 1).
"""
import numpy as np
import pytest

import kv_ref
import tree_ref
from test_kv4_gpu import _built, make  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def tables(rows, rot, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.uniform(-np.pi, np.pi, (rows, rot // 2))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def sections(half, axes):
    return [min(axes - 1, j * axes // half) for j in range(half)]


ROPE = [
    # lens, nq, hq, hkv, D, page, rot, axes, interleaved
    ([1], [1], 1, 1, 64, 16, 64, None, False),
    ([40, 7, 100], [3, 7, 1], 8, 2, 128, 16, 128, None, False),
    ([40, 7, 100], [3, 7, 1], 8, 2, 128, 32, 128, None, True),
    ([33, 64], [33, 20], 6, 3, 64, 48, 64, sections(32, 3), False),
    ([33, 64], [33, 20], 5, 5, 64, 16, 32, sections(16, 2), True),         # half of the channels
    ([200, 0, 90], [150, 0, 90], 14, 2, 128, 64, 128, [j % 3 for j in range(64)], False),  # axes in turn
    ([61], [61], 3, 1, 128, 16, 32, [j % 4 for j in range(16)], True),
    ([61], [30], 3, 1, 128, 16, 48, None, False),                          # 24 pairs
    ([61], [30], 2, 2, 64, 16, 8, None, False),                            # one chunk a half
    ([500, 1200], [500, 1100], 32, 8, 128, 128, 128, [0] * 16 + [1] * 24 + [2] * 24, False),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,rot,axes,interleaved", ROPE)
def test_rotates_and_appends(lens, nq, hq, hkv, D, page, rot, axes, interleaved):
    import w4a16_mixed_precision_gb300 as w4
    _, _, cache, batch, _ = make(lens, nq, hkv, D, page, seed=sum(lens))
    T, rows = sum(nq), 777
    rng = np.random.default_rng(T)
    qkv = rng.standard_normal((T, hq + 2 * hkv, D)).astype(np.float16)
    cos, sin = tables(rows, rot)
    n_axes = 1 if axes is None else max(axes) + 1
    positions = rng.integers(0, rows, (n_axes, T)).astype(np.int32)
    positions[:, 0], positions[:, -1] = 0, rows - 1
    rope = w4.Kv4Rope(cuda(cos), cuda(sin), axes=axes, interleaved=interleaved)
    ws = w4.Kv4Workspace(batch, hq, cache)
    dev = cuda(qkv)
    q, k, v = dev.split([hq, hkv, hkv], dim=1)
    before = dev.clone()
    dp = cuda(positions) if n_axes > 1 else cuda(positions[0])
    out = w4.kv4_rope_append(q, k, v, dp, rope, cache, batch, ws)
    assert w4.device_status(ws) == 0 and torch.equal(dev, before)
    pairs = axes or [0] * (rot // 2)
    q32, q64 = tree_ref.rotate(qkv[:, :hq], positions, cos, sin, pairs, interleaved)
    k32, _ = tree_ref.rotate(qkv[:, hq:hq + hkv], positions, cos, sin, pairs, interleaved)
    got = out.cpu().numpy()
    assert np.array_equal(got, q32)
    x = np.abs(qkv[:, :hq].astype(np.float64)).max()
    assert (np.abs(got - q64) <= 2.0 ** -11 * np.abs(q64) + 3 * 2.0 ** -24 * 2 * x + 2.0 ** -25).all()
    kr, vr = w4.kv4_read(cache, batch, ws)
    assert np.array_equal(kr.cpu().numpy(), kv_ref.values(k32).astype(np.float16))
    assert np.array_equal(vr.cpu().numpy(), kv_ref.values(qkv[:, hq + hkv:]).astype(np.float16))
    # the same bytes as kv4_append of the rotated keys, and in place
    bytes_ = cache.buf.clone()
    w4.kv4_append(cuda(k32), v, cache, batch, ws)
    assert torch.equal(cache.buf, bytes_)
    assert w4.kv4_rope_append_into(q, k, v, dp, rope, cache, batch, ws, q) is q
    assert np.array_equal(q.cpu().numpy(), q32) and torch.equal(dev[:, hq:], before[:, hq:])


def test_far_positions_from_theta():
    """Angles are taken in 64 bits: at a position of 2^20 the table is as near to cos and sin as fp32 is."""
    import w4a16_mixed_precision_gb300 as w4
    n = (1 << 20) + 5
    rope = w4.Kv4Rope.from_theta(128, n, theta=1e6)
    at = np.array([1, 1000, n - 1])
    angle = at[:, None] * 1e6 ** (-np.arange(0, 128, 2) / 128)
    t = rope.table[cuda(at)].cpu().numpy()
    # the angle's own error in 64 bits, 2^-52 of up to 2^20, then the rounding to fp32
    assert np.abs(t[..., 0] - np.cos(angle)).max() <= 2.0 ** -24 and np.abs(t[..., 1] - np.sin(angle)).max() <= 2.0 ** -24


def test_infinities_zeros_and_overflow():
    """A key that holds or becomes infinite is NaN in the cache, others are not touched by it; queries as they come."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [20], [20], 2, 2, 64, 16
    _, _, cache, batch, _ = make(lens, nq, hkv, D, page, seed=1)
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((20, 2, D)).astype(np.float16) for _ in range(3))
    k[3, 1, 5] = np.inf
    k[4, 0, 0], k[4, 0, 32] = 60000, 60000   # the sum of both passes fp16's range
    k[5, 0] = 0
    q[6, 0, 1], q[7, 1, 2] = np.nan, -np.inf
    cos, sin = np.full((4, 32), 0.7071067, np.float32), np.full((4, 32), 0.7071067, np.float32)
    rope = w4.Kv4Rope(cuda(cos), cuda(sin))
    ws = w4.Kv4Workspace(batch, hq, cache)
    out = w4.kv4_rope_append(cuda(q), cuda(k), cuda(v), torch.zeros(20, dtype=torch.int32, device="cuda"), rope, cache, batch, ws)
    assert w4.device_status(ws) == 0
    pos = np.zeros((1, 20), np.int32)
    assert np.array_equal(out.cpu().numpy(), tree_ref.rotate(q, pos, cos, sin, [0] * 32, False)[0], equal_nan=True)
    k32 = tree_ref.rotate(k, pos, cos, sin, [0] * 32, False)[0]
    assert np.isinf(k32[4, 0]).any()
    kr, vr = w4.kv4_read(cache, batch, ws)
    assert np.array_equal(kr.cpu().numpy(), kv_ref.values(k32).astype(np.float16), equal_nan=True)
    assert np.array_equal(vr.cpu().numpy(), kv_ref.values(v).astype(np.float16))


def test_rows_behind_the_last_request_and_bad_entries():
    """Padded rows are left alone whatever their positions; a position outside the table, a bad page and a length that
    does not fit are reported, and other tokens are right."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [40, 30], [6, 5], 4, 2, 128, 16
    _, _, cache, batch, _ = make(lens, nq, hkv, D, page, seed=3)
    T, rows = 11 + 3, 50
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((T, h, D)).astype(np.float16) for h in (hq, hkv, hkv))
    cos, sin = tables(rows, D)
    rope = w4.Kv4Rope(cuda(cos), cuda(sin))
    positions = rng.integers(0, rows, T).astype(np.int32)
    positions[11:] = (-5, rows, 1 << 30)
    good = w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, T, 6)
    ws = w4.Kv4Workspace(good, hq, cache)
    out = torch.full((T, hq, D), 3.0, dtype=torch.float16, device="cuda")
    run = lambda b, p: w4.kv4_rope_append_into(cuda(q), cuda(k), cuda(v), cuda(p), rope, cache, b, ws, out)  # noqa: E731
    run(good, positions)
    assert w4.device_status(ws) == 0
    ref = tree_ref.rotate(q, np.clip(positions, 0, rows - 1)[None], cos, sin, [0] * 64, False)[0]
    assert np.array_equal(out[:11].cpu().numpy(), ref[:11]) and (out[11:] == 3).all()
    clean = cache.buf.clone()
    for wrong in (rows, -1, -(1 << 31)):
        bad = positions.copy()
        bad[2] = wrong
        out.fill_(3.0)
        run(good, bad)
        assert w4.device_status(ws) == 7
        assert (out[2] == 3).all() and np.array_equal(out[3:11].cpu().numpy(), ref[3:11])
        assert torch.equal(cache.buf, clean)
    table = batch.page_table.clone()
    table[1] = cache.n_pages
    run(w4.Kv4Batch(table, batch.lengths, batch.q_start, T, 6), positions)
    assert w4.device_status(ws) == 7 and torch.equal(cache.buf, clean)
    short = batch.lengths.clone()
    short[1] = 3
    before = cache.buf.clone()
    run(w4.Kv4Batch(batch.page_table, short, batch.q_start, T, 6), positions)
    assert w4.device_status(ws) == 7
    assert np.array_equal(out[:6].cpu().numpy(), ref[:6]) and not torch.equal(cache.buf, before)  # the last three tokens fit


def test_streams_and_graphs():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [100, 30], [2, 1], 8, 2, 128, 64
    _, _, cache, batch, _ = make(lens, nq, hkv, D, page, seed=5)
    rng = np.random.default_rng(6)
    q, k, v = (cuda(rng.standard_normal((3, h, D)).astype(np.float16)) for h in (hq, hkv, hkv))
    cos, sin = tables(128, D)
    rope = w4.Kv4Rope(cuda(cos), cuda(sin))
    ws = w4.Kv4Workspace(batch, hq, cache)
    positions = torch.tensor([5, 6, 99], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.kv4_rope_append_into(q, k, v, positions, rope, cache, batch, ws, out)
    positions.copy_(torch.tensor([127, 0, 1], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert w4.device_status(ws) == 0
    pos = np.array([[127, 0, 1]])
    assert np.array_equal(out.cpu().numpy(), tree_ref.rotate(q.cpu().numpy(), pos, cos, sin, [0] * 64, False)[0])


def test_refusals():
    import w4a16_mixed_precision_gb300 as w4
    k_, v_, cache, batch, _ = make([40], [2], 2, 128, 16, seed=14)
    ws = w4.Kv4Workspace(batch, 4, cache)
    q = torch.zeros((2, 4, 128), dtype=torch.float16, device="cuda")
    k, pos = q[:, :2], torch.zeros(2, dtype=torch.int32, device="cuda")
    cos, sin = (cuda(x) for x in tables(10, 128))
    rope = w4.Kv4Rope(cos, sin)
    two = w4.Kv4Rope(cos, sin, axes=[0, 1] * 32)
    go = lambda q=q, k=k, v=k, p=pos, rope=rope, out=q: w4.kv4_rope_append_into(q, k, v, p, rope, cache, batch, ws, out)  # noqa: E731
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(k=q), dict(v=q[:, :1]), dict(out=q[:, :2]),
                dict(out=q.float()), dict(p=pos.long()), dict(p=pos[:1]), dict(p=pos.cpu()), dict(rope=two),
                dict(rope=two, p=pos.view(1, 2)), dict(p=torch.zeros((2, 2), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            go(**bad)
    for rot, status in ((40, 2), (130, 1)):   # no multiple of 16; more than head_dim
        c, s = (cuda(x) for x in tables(10, rot))
        with pytest.raises(w4.MarlinError) as e:
            go(rope=w4.Kv4Rope(c, s))
        assert e.value.status == status
    odd = torch.zeros((2, 4 * 128 + 4), dtype=torch.float16, device="cuda")[:, 4:].view(2, 4, 128)
    with pytest.raises(w4.MarlinError) as e:
        go(q=odd)
    assert e.value.status == 3
    for args in ((cos.double(), sin.double()), (cos.cpu(), sin.cpu()), (cos, sin[:5]), (cos[0], sin[0]), (cos[:0], sin[:0])):
        with pytest.raises(ValueError):
            w4.Kv4Rope(*args)
    for axes in ([0] * 63, [0, 4] * 32, [-1] * 64):
        with pytest.raises(ValueError):
            w4.Kv4Rope(cos, sin, axes=axes)
    assert w4.device_status(ws) == 0
