"""Tree attention of many rows over long caches, where a CTA's stripe has more blocks of an item than it sums in tensor
memory at a time: pieces that follow each other on the same rows, items that end inside a stripe after several, a
stripe with the end of an item, whole ones and the beginning of another.  And how precise the results are, in root mean
square.

Tolerances.  Element by element those of test_kv4_tree_gpu.py.  The mean over tokens is small beside each value, so that
what is lost on the way shows in root mean square: the kernel for many rows rounds every p s (a probability times its
value vector's scale) to fp16 and the output to fp16, and may have at most 1.1 times the error of just that, in 64 bits
otherwise (fp32 sums of n terms of random signs leave sqrt(n) 2^-24, 3e-5 of a term at 300,000, a tenth of fp16's 2^-11
on each term).  The kernel for few rows holds p s in two fp16 numbers, 2^-22: at most 1.1 times the output's rounding.
"""
import numpy as np
import pytest

import kv_ref
import kv_torch
import tree_ref
from test_kv4_gpu import _built, make, split  # noqa: F401
from test_kv4_tree_gpu import near

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

PIECE, ROWS, BLOCK = 56, 256, 64   # blocks of a piece, rows of an item, tokens of a block


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def blocks_of(length, n, window):
    lo = max(0, length - n - window) // BLOCK if window else 0
    return max(1, -(-length // BLOCK) - lo)


def most_blocks_a_cta(lens, nq, hq, hkv, window):
    """(blocks of the longest item, blocks of a stripe, items, SMs)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    items = [-(-n * (hq // hkv) // ROWS) * hkv for n in nq]
    blocks = [blocks_of(length, n, window) for length, n in zip(lens, nq)]
    total = sum(i * b for i, b in zip(items, blocks))
    return max(blocks), total / sms, sum(items), sms


def widest(v):
    """The vectors with the largest value and the widest range, which the tolerances go by."""
    x = kv_torch.values(v).flatten(0, 1)
    return x[torch.stack([x.abs().amax(-1).argmax(), (x.amax(-1) - x.amin(-1)).argmax()])].cpu().numpy()


def inputs(lens, nq, hq, hkv, D, page, seed, grow=0.0):
    """Keys and values of whole histories on the GPU, appended; grow: scores rise by so much towards the end."""
    import w4a16_mixed_precision_gb300 as w4
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    per = [-(-n // page) for n in lens]
    order = torch.randperm(sum(per) + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(per):
        table[b, :n] = order[sum(per[:b]):sum(per[:b + 1])]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    start = lambda n: i32([sum(n[:b]) for b in range(len(n) + 1)])  # noqa: E731
    H = sum(lens)
    k, v, q = normal(H, hkv, D), normal(H, hkv, D), normal(sum(nq), hq, D)
    if grow:  # channels 0 to 15 of q are 1, of k they grow: 16 of them give the score
        q[..., :16] = 1
        at = torch.cat([torch.arange(n, device="cuda") / n for n in lens])
        k[..., :16] = (grow * D ** 0.5 / 16 * at)[:, None, None].half()
    cache = w4.Kv4Cache(len(order), hkv, D, page)
    hist = w4.Kv4Batch(table, i32(lens), start(lens), H, max(lens))
    batch = w4.Kv4Batch(table, i32(lens), start(nq), sum(nq), max(nq))
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(k, v, cache, hist, ws)
    rng = np.random.default_rng(seed)
    see = [tree_ref.sees(tree_ref.random_parents(n, rng)) for n in nq]
    words = -(-max(nq) // 32)
    return q, k, v, cache, batch, ws, see, cuda(np.concatenate([tree_ref.bits(s, words) for s in see]))


def test_the_torch_reference_is_kv_refs():
    rng = np.random.default_rng(0)
    for n, hq, hkv, D, window in ((5, 4, 2, 64, 0), (30, 2, 1, 128, 20)):
        q, k, v = (rng.standard_normal(s).astype(np.float16) for s in ((n, hq, D), (90, hkv, D), (90, hkv, D)))
        k[3, 0] = 0.5
        see = tree_ref.sees(tree_ref.random_parents(n, rng))
        assert np.array_equal(kv_torch.values(cuda(k)).cpu().numpy(), kv_ref.values(k))
        ref = tree_ref.attention(q, kv_ref.values(k), kv_ref.values(v), see, D ** -0.5, window)
        got = kv_torch.attention(cuda(q), cuda(k), cuda(v), cuda(see), D ** -0.5, window).cpu().numpy()
        assert np.abs(got - ref).max() <= 1e-12


PIECES = [
    # lens, nq, hq, hkv, D, page, window, how far scores grow
    ([100000], [9], 64, 8, 128, 64, 0, 0.0),                                  # stripes of 82 blocks cut items of 1563
    ([150001], [40], 16, 8, 64, 128, 0, 0.0),                                 # one tile of an item alone
    ([64 * (57 + 83 * i % 84) - i for i in range(40)], [9 + i % 30 for i in range(40)], 64, 8, 128, 64, 0, 0.0),  # 57 to 140 blocks
    ([64 * (57 + 47 * i % 84) - 3 * i for i in range(45)], [35 + i % 3 for i in range(45)], 16, 8, 64, 16, 0, 0.0),
    ([9000 + 401 * i for i in range(40)], [20] * 40, 32, 8, 128, 32, 5000, 0.0),   # windowed
    ([120000], [33], 32, 8, 128, 64, 0, 20.0),                               # the reference moves from piece to piece
    ([64 * (140 - i % 30) for i in range(40)], [17] * 40, 32, 8, 64, 64, 0, 20.0),
    ([150000, 100, 40], [70, 90, 3], 8, 8, 128, 64, 0, 0.0),                  # both kernels
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window,grow", PIECES)
def test_pieces(lens, nq, hq, hkv, D, page, window, grow):
    import w4a16_mixed_precision_gb300 as w4
    longest, stripe, items, sms = most_blocks_a_cta(lens, nq, hq, hkv, window)
    # a CTA has more blocks of one item than a piece, and no CTA takes an item whole
    assert longest > PIECE and stripe > PIECE and (items > sms or longest > stripe + 20)
    q, k, v, cache, batch, ws, see, tree = inputs(lens, nq, hq, hkv, D, page, sum(lens) % 1000, grow)
    y = w4.kv4_tree_attention(q, cache, batch, tree, ws, window=window)
    for _ in range(5):
        assert torch.equal(w4.kv4_tree_attention(q, cache, batch, tree, ws, window=window), y)
    assert w4.device_status(ws) == 0
    t = h = 0
    for length, n, s in zip(lens, nq, see):
        kk, vv = k[h:h + length], v[h:h + length]
        ref = kv_torch.attention(q[t:t + n], kk, vv, cuda(s), D ** -0.5, window)
        near(y[t:t + n].cpu().numpy(), ref.cpu().numpy(), widest(vv), n * hq // hkv)
        t, h = t + n, h + length


@pytest.mark.parametrize("length,nq,hq,hkv,D", [
    (300001, 9, 64, 8, 128),   # 247 blocks of an item a CTA on 152 SMs
    (260000, 17, 32, 8, 64),
    (20000, 25, 24, 8, 128),
])
def test_many_rows_lose_what_rounding_p_s_loses(length, nq, hq, hkv, D):
    import w4a16_mixed_precision_gb300 as w4
    q, k, v, cache, batch, ws, see, tree = inputs([length], [nq], hq, hkv, D, 64, nq)
    y = w4.kv4_tree_attention(q, cache, batch, tree, ws)
    assert w4.device_status(ws) == 0
    see = cuda(see[0])
    ref = kv_torch.attention(q, k, v, see, D ** -0.5)
    sim = kv_torch.attention(q, k, v, see, D ** -0.5, rounded=True).half()
    lost, may = kv_torch.rms(y - ref), kv_torch.rms(sim - ref)
    print(f"{lost / kv_torch.rms(ref):.3e} of the result, rounding p s and the output {may / kv_torch.rms(ref):.3e}")
    assert lost <= 1.1 * may


@pytest.mark.parametrize("length,nq,hq,hkv,D", [(5000, 8, 48, 8, 128), (5000, 7, 64, 8, 128), (9000, 16, 8, 2, 64), (900, 50, 2, 2, 64)])
def test_trees_of_up_to_64_rows_a_key_head_lose_what_rounding_the_output_loses(length, nq, hq, hkv, D):
    """As kv4_attention, whatever the number of their rows."""
    import w4a16_mixed_precision_gb300 as w4
    assert 48 <= nq * hq // hkv <= 64
    q, k, v, cache, batch, ws, see, tree = inputs([length], [nq], hq, hkv, D, 64, nq)
    y = w4.kv4_tree_attention(q, cache, batch, tree, ws)
    assert w4.device_status(ws) == 0
    ref = kv_torch.attention(q, k, v, cuda(see[0]), D ** -0.5)
    lost, may = kv_torch.rms(y - ref), kv_torch.rms(ref.half() - ref)
    print(f"{lost / kv_torch.rms(ref):.3e} of the result, rounding the output {may / kv_torch.rms(ref):.3e}")
    assert lost <= 1.1 * may
