"""Rotary positions with the append where a warp has several steps (four tokens, 1 KB of their heads each): angles and
places that are kept from step to step, runs that begin in the middle of the tokens' heads or end before their keys.
Queries bit for bit products and sums rounded one by one (elementary operations of torch), the cache byte for byte what
kv4_append makes of keys rotated so.
"""
import pytest

from test_kv4_gpu import _built, make  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def steps_a_warp(T, hq, hkv, D):
    """Steps of all tokens over the warps that are on the card at a time (3 CTAs of 8 an SM); a step each up to 2."""
    vectors = 512 // D
    steps = -(-T // 4) * (-(-hq // vectors) + -(-2 * hkv // vectors))
    return steps / (torch.cuda.get_device_properties(0).multi_processor_count * 24)


def rotate(x, positions, cos, sin, axes, interleaved):
    """x fp16 [T, H, D] -> fp16."""
    pair = torch.arange(len(axes), device="cuda")
    at = positions.long()[torch.tensor(axes, device="cuda")].t()        # [T, pairs]
    c, s = cos[at, pair][:, None], sin[at, pair][:, None]
    half, f, out = len(axes), x.float(), x.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    x1, x2 = f[..., first], f[..., second]
    a, b = x1 * c, x2 * s
    d, e = x2 * c, x1 * s
    out[..., first], out[..., second] = (a - b).half(), (d + e).half()
    return out


RUNS = [
    # lens, nq, hq, hkv, D, page, rot, axes, interleaved
    ([4001], [4001], 32, 8, 128, 64, 128, None, False),
    ([5000, 300, 2803], [4990, 1, 2790], 32, 8, 128, 16, 128, [0] * 16 + [1] * 24 + [2] * 24, False),
    ([3001, 0, 2002], [3001, 0, 2000], 64, 8, 128, 128, 64, [j % 3 for j in range(32)], True),     # axes in turn
    ([6007, 5, 3003], [6001, 5, 3003], 32, 8, 64, 48, 64, None, True),
    ([9001], [9001], 20, 5, 64, 32, 32, [j % 4 for j in range(16)], False),                       # no whole steps
    ([40] * 300, [39] * 300, 7, 7, 128, 16, 128, None, False),
]


def setup(lens, nq, hq, hkv, D, page, rot, axes, interleaved, seed):
    import w4a16_mixed_precision_gb300 as w4
    _, _, cache, batch, _ = make(lens, nq, hkv, D, page, seed=seed)
    g = torch.Generator("cuda").manual_seed(seed)
    T, rows = sum(nq), 5000
    qkv = torch.randn((T, hq + 2 * hkv, D), generator=g, device="cuda", dtype=torch.float16)
    angle = torch.rand((rows, rot // 2), generator=g, device="cuda", dtype=torch.float64) * 6.3
    cos, sin = angle.cos().float(), angle.sin().float()
    pairs = axes or [0] * (rot // 2)
    positions = torch.randint(0, rows, (max(pairs) + 1, T), generator=g, device="cuda", dtype=torch.int32)
    rope = w4.Kv4Rope(cos, sin, axes=axes, interleaved=interleaved)
    return cache, batch, w4.Kv4Workspace(batch, hq, cache), qkv, positions, rope, lambda x, p: rotate(x, p, cos, sin, pairs, interleaved)


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,rot,axes,interleaved", RUNS)
def test_runs_of_steps(lens, nq, hq, hkv, D, page, rot, axes, interleaved):
    import w4a16_mixed_precision_gb300 as w4
    assert steps_a_warp(sum(nq), hq, hkv, D) > 2
    cache, batch, ws, qkv, positions, rope, rotated = setup(lens, nq, hq, hkv, D, page, rot, axes, interleaved, seed=len(lens) + D)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    before, old = qkv.clone(), cache.buf.clone()
    out = w4.kv4_rope_append(q, k, v, positions, rope, cache, batch, ws)
    assert w4.device_status(ws) == 0 and torch.equal(qkv, before)
    want = rotated(q, positions)
    assert torch.equal(out, want)
    got = cache.buf.clone()
    cache.buf.copy_(old)
    w4.kv4_append(rotated(k, positions), v, cache, batch, ws)
    assert torch.equal(got, cache.buf) and not torch.equal(got, old)
    cache.buf.copy_(old)
    assert w4.kv4_rope_append_into(q, k, v, positions, rope, cache, batch, ws, q) is q
    assert torch.equal(q, want) and torch.equal(qkv[:, hq:], before[:, hq:]) and torch.equal(cache.buf, got)
    assert w4.device_status(ws) == 0


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 128), (24, 8, 64)])
def test_bad_entries_in_the_middle_of_runs(hq, hkv, D):
    """Positions outside the table and a page that does not exist, among thousands of tokens: reported, those tokens left
    out (their queries alone rotated where the page is bad), all others right; rows behind the last request are left alone."""
    import w4a16_mixed_precision_gb300 as w4
    n, pad, page, D_ = 9001, 37, 64, D
    cache, batch, _, qkv, positions, rope, rotated = setup([n], [n], hq, hkv, D_, page, D_, None, False, seed=D)
    T = n + pad
    more = torch.randn((pad, hq + 2 * hkv, D), device="cuda", dtype=torch.float16)
    q, k, v = torch.cat([qkv, more]).split([hq, hkv, hkv], dim=1)
    padded = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    padded[:n] = positions[0]
    table = batch.page_table.clone()
    table[0, 70] = cache.n_pages                                # tokens 4480 to 4543
    bad = torch.tensor([0, 1, 2, 3, 801, 4000, 4003, 6002, n - 1], device="cuda")
    wrong = padded.clone()
    wrong[bad] = torch.tensor([5000, -1, 1 << 30, -(1 << 31), 5001, 5000, 5000, -7, 5000], dtype=torch.int32, device="cuda")
    whole = w4.Kv4Batch(batch.page_table, batch.lengths, batch.q_start, T, n)
    ws = w4.Kv4Workspace(whole, hq, cache)
    first = torch.randn((T, hkv, D), device="cuda", dtype=torch.float16)
    w4.kv4_append(first, first, cache, whole, ws)
    old = w4.kv4_read(cache, whole, ws)
    out = torch.full((T, hq, D), 3.0, device="cuda", dtype=torch.float16)
    assert w4.device_status(ws) == 0 and steps_a_warp(T, hq, hkv, D) > 2
    w4.kv4_rope_append_into(q, k, v, wrong, rope, cache, w4.Kv4Batch(table, batch.lengths, batch.q_start, T, n), ws, out)
    assert w4.device_status(ws) == 7
    want = rotated(q[:n], positions)
    want[bad] = 3.0
    assert torch.equal(out[:n], want) and bool((out[n:] == 3).all())
    got = w4.kv4_read(cache, whole, ws)
    left = torch.zeros(n, dtype=torch.bool, device="cuda")
    left[bad] = True
    left[70 * page:71 * page] = True
    w4.kv4_append(torch.cat([rotated(k[:n], positions), k[n:]]), v, cache, whole, ws)
    new = w4.kv4_read(cache, whole, ws)
    assert w4.device_status(ws) == 0
    for a, b, c in zip(got, old, new):
        assert torch.equal(a[:n][left], b[:n][left]) and torch.equal(a[:n][~left], c[:n][~left])
