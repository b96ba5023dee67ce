"""The 4-bit paged cache on the GPU: what is written reads back bit for bit as
the format defines it, and attention over it against a plain implementation in
64 bits.

Tolerance of attention, derived: the output is rounded once to fp16 (half an
ulp, 2^-11 |y|).  A score in units of log2 is a sum of D products q c whose
magnitudes add up to a few tens; fp32 accumulation over D/16 steps leaves an
absolute error of at most 2^-13 in it, so every probability is off by at most
2^-13 of itself and so is their sum: 2 * 2^-13 * max |v| for the quotient.
"""
import numpy as np
import pytest

import kv_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def close(y, ref, v):
    """Within the tolerance above; NaN exactly where the reference has it."""
    y = np.asarray(y, np.float64)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    ok = ~np.isnan(ref)
    top = np.nanmax(np.abs(v)) if v.size else 0.0
    err = np.abs(y - ref)[ok]
    tol = (2.0 ** -11 * np.abs(ref) + 2.0 ** -12 * top + 2.0 ** -24)[ok]
    assert (err <= tol).all(), f"max error {err.max()}, {(err / tol).max():.2f} of the tolerance"


def make(lens, nq, hkv, D, page, seed, spread=1.0):
    """History and batch: k, v fp16 numpy per request, a cache filled by one append, the batch of the new tokens."""
    import w4a16_mixed_precision_gb300 as w4
    rng = np.random.default_rng(seed)
    dev = torch.device("cuda", 0)
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + 2
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(max(per), 1)), -1, np.int32)  # unused entries are not valid pages
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    H = sum(lens)
    k = (spread * rng.standard_normal((H, hkv, D))).astype(np.float16)
    v = (spread * rng.standard_normal((H, hkv, D))).astype(np.float16)
    k[:, :, :3] += np.float16(2.5)
    cache = w4.Kv4Cache(n_pages, hkv, D, page)
    cache.buf.random_(0, 256)  # slots that nobody wrote hold anything, NaN scales among it
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    starts = lambda n: t(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))  # noqa: E731
    dt, dl = t(table), t(np.array(lens, np.int32))
    batch = w4.Kv4Batch(dt, dl, starts(nq), sum(nq), max(nq))
    hist = w4.Kv4Batch(dt, dl, starts(lens), H, max(lens))
    return k, v, cache, batch, hist


def split(x, lens):
    return np.split(x, np.cumsum(lens)[:-1])


APPEND = [
    # lens, hkv, D, page
    ([1], 1, 64, 16),
    ([5, 0, 33], 2, 128, 16),
    ([17, 64, 63, 1], 8, 128, 32),
    ([130], 3, 64, 48),
    ([256, 100], 4, 128, 128),
]


@pytest.mark.parametrize("lens,hkv,D,page", APPEND)
def test_append_reads_back_as_the_format_says(lens, hkv, D, page):
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make(lens, lens, hkv, D, page, seed=len(lens) + D)
    # constant vectors, tiny and huge ranges, subnormals, zeros; infinities and NaN
    k[0, 0] = 1.25
    k[-1, 0, :] = 0
    v[0, 0, :] = np.linspace(-65504, 65504, D).astype(np.float16)
    v[-1, 0, :] = (np.arange(D) * 2.0 ** -24).astype(np.float16)
    if k.shape[0] > 3:
        k[2, -1, 5] = np.inf
        v[3, 0, D - 1] = np.nan
        k[3, 0, 0], k[3, 0, 1] = np.inf, -np.inf
    ws = w4.Kv4Workspace(hist, hkv, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    kr, vr = w4.kv4_read(cache, hist, ws)
    assert w4.device_status(ws) == 0
    for got, x in ((kr, k), (vr, v)):
        ref = kv_ref.values(x).astype(np.float16)
        got = got.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = ~np.isnan(ref)
        assert np.array_equal(got[ok], ref[ok])


def test_append_token_by_token_equals_one_append_and_strided_views():
    """Tokens appended one at a time, from views of one QKV product, give the bytes of one append."""
    import w4a16_mixed_precision_gb300 as w4
    lens, hkv, D, page = [37, 20], 2, 128, 16
    k, v, cache, _, hist = make(lens, lens, hkv, D, page, seed=3)
    ws = w4.Kv4Workspace(hist, hkv, cache)
    cache.buf.zero_()
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    one = cache.buf.clone()
    cache.buf.zero_()
    ks, vs = split(k, lens), split(v, lens)
    for i in range(max(lens)):
        now = [b for b in range(2) if i < lens[b]]
        qkv = np.zeros((len(now), 3, hkv, D), np.float16)
        for r, b in enumerate(now):
            qkv[r, 1], qkv[r, 2] = ks[b][i], vs[b][i]
        dev = torch.from_numpy(qkv).cuda()
        start = np.zeros(3, np.int32)
        for b in range(2):
            start[b + 1] = start[b] + (b in now)
        cur = np.array([min(i + 1, n) for n in lens], np.int32)
        batch = w4.Kv4Batch(hist.page_table, torch.from_numpy(cur).cuda(), torch.from_numpy(start).cuda(), len(now), 1)
        w4.kv4_append(dev[:, 1], dev[:, 2], cache, batch, ws)
    assert w4.device_status(ws) == 0
    assert torch.equal(cache.buf, one)


ATTENTION = [
    # lens, nq, hq, hkv, D, page, window
    ([1], [1], 1, 1, 64, 16, 0),                          # one token, one key
    ([1, 2, 15, 16, 17], [1] * 5, 4, 2, 128, 16, 0),      # granule ends
    ([300], [1], 8, 8, 128, 64, 0),                       # one head per key head
    ([1000, 3, 257], [1, 1, 1], 16, 2, 128, 32, 0),       # 8 rows
    ([700, 90], [1, 1], 15, 5, 64, 48, 0),                # 3 rows, pages of three granules
    ([513, 40], [1, 1], 32, 2, 128, 128, 0),              # 16 rows
    ([400], [1], 40, 2, 64, 16, 0),                       # 20 rows: two blocks
    ([600, 130], [5, 2], 8, 2, 128, 16, 0),               # proposed tokens, ragged
    ([90, 33], [90, 7], 4, 4, 64, 32, 0),                 # a whole prompt beside a few tokens
    ([200, 64], [70, 64], 6, 2, 128, 64, 0),
    ([500, 20, 77], [1, 1, 1], 8, 2, 128, 16, 33),        # window, shorter than a request and not
    ([300, 100], [9, 100], 4, 2, 64, 16, 17),             # window inside the new tokens
    ([200], [3], 8, 1, 128, 64, 1),                       # a token sees itself alone
    ([64, 0, 5], [1, 0, 1], 4, 2, 128, 16, 0),            # a request without tokens
    ([20000], [1], 8, 1, 128, 64, 0),                     # split over many CTAs
    ([9000], [2], 16, 2, 64, 256, 5000),
    # many query rows per key head: tiles of 128 rows, blocks of 64 tokens
    ([65], [65], 1, 1, 64, 16, 0),                        # one row more than the streaming kernel takes
    ([128], [128], 2, 2, 128, 64, 0),                     # exactly one tile
    ([129, 1, 300], [129, 1, 300], 3, 3, 128, 32, 0),     # tiles of one row; one request beside them
    ([500], [100], 7, 1, 128, 16, 0),                     # a later part of a prompt, 7 heads share a key head
    ([777], [777], 4, 1, 64, 48, 0),
    ([1000], [300], 4, 2, 128, 128, 100),                 # window shorter than a block pair
    ([400], [400], 2, 1, 64, 16, 1),                      # every token sees itself alone
    ([640, 64], [200, 64], 8, 8, 128, 64, 64),
    # many requests: more than threads of a CTA; several whole requests in a warp's stripe
    ([i * 7 % 50 + 1 for i in range(300)], [1] * 300, 4, 1, 64, 16, 0),
    ([i * 37 % 400 + 1 for i in range(60)], [1] * 60, 8, 2, 128, 32, 0),
    # whole segments for every warp: one or none of equal ones, several of unequal ones, two row groups
    ([130] * 40, [1] * 40, 8, 8, 128, 32, 0),
    ([i * 11 % 120 + 3 for i in range(100)], [1, 2, 0, 3] * 25, 32, 16, 64, 16, 0),
    ([100 + i % 3 for i in range(50)], [9] * 50, 16, 8, 128, 16, 64),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", ATTENTION)
def test_attention(lens, nq, hq, hkv, D, page, window):
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=sum(lens) + hq)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    rng = np.random.default_rng(5)
    q = rng.standard_normal((sum(nq), hq, D)).astype(np.float16)
    dq = torch.from_numpy(q).cuda()
    y = w4.kv4_attention(dq, cache, batch, ws, window=window)
    again = w4.kv4_attention(dq, cache, batch, ws, window=window)
    assert w4.device_status(ws) == 0
    assert torch.equal(y, again)
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
        close(yy, kv_ref.attention(qq, kv[b], vv[b], nq[b], D ** -0.5, window), vv[b])


LONG_PROMPTS = [
    # few items of many tokens: cut over CTAs and joined
    ([3000], [100], 7, 1, 128, 16, 0),
    ([2500, 40, 3100], [70, 40, 90], 8, 2, 64, 32, 0),
    ([4000, 2900], [150, 300], 2, 1, 128, 64, 2600),
    ([6001], [65], 16, 1, 64, 48, 0),                     # one item but a little
    # more items than SMs: a CTA for each, and CTAs without one
    ([90] * 22, [80] * 22, 8, 8, 64, 16, 0),
    ([200, 1, 75, 40] * 9, [100, 1, 75, 33] * 9, 8, 8, 128, 32, 0),
    ([300] * 40, [70] * 40, 12, 6, 64, 64, 100),
]


@pytest.mark.parametrize("lens,nq,hq,hkv,D,page,window", LONG_PROMPTS)
def test_prompts_cut_over_ctas_and_a_cta_each(lens, nq, hq, hkv, D, page, window):
    test_attention(lens, nq, hq, hkv, D, page, window)


@pytest.mark.parametrize("nq", [1, 80])
def test_long_context_is_as_accurate_as_its_rounding(nq):
    """The mean of many values is small beside each: what is lost on the way to it, in root mean square, is no
    more than rounding the result itself (2^-11 / sqrt(3) of it at most), on few rows and on tiles of 128;
    the two together are sqrt(2) times that."""
    import w4a16_mixed_precision_gb300 as w4
    lens, hq, hkv, D, page = [131001], 4, 1, 128, 64
    k, v, cache, batch, hist = make(lens, [nq], hkv, D, page, seed=30)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = np.random.default_rng(31).standard_normal((nq, hq, D)).astype(np.float16)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws).cpu().numpy().astype(np.float64)
    assert w4.device_status(ws) == 0
    some = slice(max(0, nq - 3), nq)
    ref = kv_ref.attention(q[some], kv_ref.values(k), kv_ref.values(v), some.stop - some.start, D ** -0.5)
    assert np.sqrt(((y[some] - ref) ** 2).mean()) <= 2.0 ** 0.5 * 2.0 ** -11 / 3 ** 0.5 * np.sqrt((ref ** 2).mean())


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_attention_of_small_and_large_values(spread):
    """Value scales near fp16's small numbers, and scores so peaked that one token takes all."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [3000, 100], [1, 3], 8, 2, 128, 64
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=8, spread=spread)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = np.random.default_rng(6).standard_normal((sum(nq), hq, D)).astype(np.float16)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws, scale=0.02 / spread)
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
        close(yy, kv_ref.attention(qq, kv[b], vv[b], nq[b], 0.02 / spread), vv[b])


def test_attention_nan_stays_where_it_is_seen():
    """A NaN key or value reaches the rows that see its token and no others; NaN in a query its own row."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [100, 40], [6, 3], 4, 2, 128, 16
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=9)
    k[97, 0, 3] = np.nan      # request 0, position 97, key head 0: rows of positions 97.. see it
    v[98, 1, 7] = np.inf      # position 98, key head 1
    q = np.random.default_rng(7).standard_normal((sum(nq), hq, D)).astype(np.float16)
    q[7, 2, 0] = np.nan       # request 1
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws).cpu().numpy()
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    nan = np.zeros(y.shape[:2], bool)
    nan[3:6, 0:2] = True      # positions 97, 98, 99
    nan[4:6, 2:4] = True      # positions 98, 99
    nan[7, 2] = True
    assert np.array_equal(np.isnan(y).any(-1), nan) and np.array_equal(np.isnan(y).all(-1), nan)
    for b, (qq, yy, bad) in enumerate(zip(split(q, nq), split(y, nq), split(nan, nq))):
        ref = kv_ref.attention(qq, kv[b], vv[b], nq[b], D ** -0.5)
        close(yy[~bad], ref[~bad], vv[b])


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_nan_and_large_scores(D):
    """The same on tiles of 128 rows: NaN keys, values and queries stay where they are seen; a block whose
    scores and value scales are far above the earlier ones moves the rows' references."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, page = [400], [200], 4, 2, 16
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=21)
    k[250:270] *= np.float16(30)     # scores up to a few hundred, from the fourth block on
    v[64:128] *= np.float16(1e-3)
    v[300:310] *= np.float16(200)
    k[390, 0, 3] = np.nan
    v[395, 1, 7] = np.inf
    q = np.random.default_rng(22).standard_normal((sum(nq), hq, D)).astype(np.float16)
    q[17, 2, 0] = np.nan
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws).cpu().numpy()
    assert w4.device_status(ws) == 0
    nan = np.zeros(y.shape[:2], bool)
    nan[190:, 0:2] = True
    nan[195:, 2:4] = True
    nan[17, 2] = True
    assert np.array_equal(np.isnan(y).any(-1), nan) and np.array_equal(np.isnan(y).all(-1), nan)
    vals = kv_ref.values(v)
    ref = kv_ref.attention(q, kv_ref.values(k), vals, 200, D ** -0.5)
    # by how much the seen values can move a row: the larger scores' fp32 error grows with them
    mag = np.abs(q.astype(np.float64)).sum(-1) * 15 * np.abs(k[:390].astype(np.float64)).max() * D ** -0.5
    tol = (2.0 ** -11 * np.abs(ref) + (2.0 ** -12 + 2.0 ** -20 * mag[:, :, None]) * np.abs(vals[:390]).max() + 2.0 ** -24)
    assert (np.abs(y - ref)[~nan] <= tol[~nan]).all()


def test_bad_entries_are_reported_and_not_followed():
    """Page numbers, lengths and starts out of range: MARLIN_ERR_BOUNDS, the context stays usable, and
    other requests' rows are right."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [50, 60], [1, 1], 4, 2, 128, 16
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=10)
    ws = w4.Kv4Workspace(batch, hq, cache)
    dk, dv = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    w4.kv4_append(dk, dv, cache, hist, ws)
    q = np.random.default_rng(8).standard_normal((2, hq, D)).astype(np.float16)
    dq = torch.from_numpy(q).cuda()
    ref = kv_ref.attention(q[:1], kv_ref.values(k)[:50], kv_ref.values(v)[:50], 1, D ** -0.5)
    good = batch.page_table.clone()
    for change in ("page", "negative page", "length", "negative length", "start"):
        table, length, start = good.clone(), batch.lengths.clone(), batch.q_start.clone()
        if change == "page":
            table[1, 2] = cache.n_pages
        elif change == "negative page":
            table[1, 0] = -7
        elif change == "length":
            length[1] = good.shape[1] * page + 1
        elif change == "negative length":
            length[1] = -3
        else:
            start[2] = 5
        bad = w4.Kv4Batch(table, length, start, 2, 1)
        y = w4.kv4_attention(dq, cache, bad, ws)
        assert w4.device_status(ws) == 7, change            # MARLIN_ERR_BOUNDS
        close(y[:1].cpu().numpy(), ref, kv_ref.values(v))
        before = cache.buf.clone()
        if change in ("page", "negative page"):
            bad_hist = w4.Kv4Batch(table, length, hist.q_start, hist.tokens, hist.max_q)
            w4.kv4_append(dk, dv, cache, bad_hist, ws)
            assert w4.device_status(ws) == 7, change
            assert torch.equal(cache.buf, before)           # the same values again, and nothing elsewhere
    y = w4.kv4_attention(dq, cache, batch, ws)
    assert w4.device_status(ws) == 0
    close(y[:1].cpu().numpy(), ref, kv_ref.values(v))


def test_more_new_tokens_than_the_length_gives_empty_rows():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [20], [20], 4, 2, 64, 16
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=11)
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = np.random.default_rng(9).standard_normal((23, hq, D)).astype(np.float16)
    start = torch.tensor([0, 23], dtype=torch.int32, device="cuda")
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, w4.Kv4Batch(batch.page_table, batch.lengths, start, 23, 23),
                         ws).cpu().numpy()
    assert w4.device_status(ws) == 7
    assert (y[:3] == 0).all()
    close(y[3:], kv_ref.attention(q[3:], kv_ref.values(k), kv_ref.values(v), 20, D ** -0.5), kv_ref.values(v))


def test_offsets_beyond_32_bits():
    """A cache of more than 4 GiB: the last page's granules are found."""
    import w4a16_mixed_precision_gb300 as w4
    hkv, D, page = 8, 128, 1024
    n_pages = (5 << 30) // (hkv * page * (D + 8)) + 1
    cache = w4.Kv4Cache(n_pages, hkv, D, page)
    rng = np.random.default_rng(12)
    n = 40
    k = rng.standard_normal((n, hkv, D)).astype(np.float16)
    v = rng.standard_normal((n, hkv, D)).astype(np.float16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    hist = w4.Kv4Batch(i([n_pages - 1]), i(n), i(0, n), n, n)
    ws = w4.Kv4Workspace(hist, hkv, cache)
    w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
    q = rng.standard_normal((1, hkv, D)).astype(np.float16)
    y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, w4.Kv4Batch(hist.page_table, hist.lengths, i(0, 1), 1, 1), ws)
    assert w4.device_status(ws) == 0
    assert int(cache.buf[:1 << 20].max()) == 0
    close(y.cpu().numpy(), kv_ref.attention(q, kv_ref.values(k), kv_ref.values(v), 1, D ** -0.5), kv_ref.values(v))


def test_on_another_stream_and_in_a_graph():
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [333, 20], [1, 1], 8, 2, 128, 64
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=13)
    ws = w4.Kv4Workspace(batch, hq, cache)
    q = np.random.default_rng(10).standard_normal((2, hq, D)).astype(np.float16)
    dk, dv, dq = (torch.from_numpy(a).cuda() for a in (k, v, q))
    out = torch.zeros((2, hq, D), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        w4.kv4_append(dk, dv, cache, hist, ws)
        w4.kv4_attention_into(dq, cache, batch, ws, out)
    s.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.kv4_attention_into(dq, cache, batch, ws, out)
    out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b in range(2):
        close(out[b:b + 1].cpu().numpy(), kv_ref.attention(q[b:b + 1], kv[b], vv[b], 1, D ** -0.5), vv[b])


def test_one_workspace_for_many_shapes():
    """What a call leaves in the workspace (arrival counts, parts) does not reach the next one."""
    import w4a16_mixed_precision_gb300 as w4
    ws = None
    for seed, (lens, nq, hq, hkv) in enumerate([([5000], [1], 8, 2), ([300, 20], [1, 1], 16, 2), ([7000, 6500], [2, 2], 16, 2),
                                                ([200], [200], 4, 2), ([5000], [1], 8, 2), ([64] * 9, [1] * 9, 8, 2)]):
        D, page = 64, 16
        k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=30 + seed)
        ws = ws or w4.Kv4Workspace(hist, 16, cache)  # the largest of them
        w4.kv4_append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), cache, hist, ws)
        q = np.random.default_rng(seed).standard_normal((sum(nq), hq, D)).astype(np.float16)
        y = w4.kv4_attention(torch.from_numpy(q).cuda(), cache, batch, ws)
        assert w4.device_status(ws) == 0
        kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
        for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
            close(yy, kv_ref.attention(qq, kv[b], vv[b], nq[b], D ** -0.5), vv[b])


def test_strided_queries():
    """Queries, keys and values as views of one QKV product."""
    import w4a16_mixed_precision_gb300 as w4
    lens, nq, hq, hkv, D, page = [90, 33], [90, 33], 8, 2, 64, 16
    k, v, cache, batch, hist = make(lens, nq, hkv, D, page, seed=40)
    T = sum(nq)
    q = np.random.default_rng(41).standard_normal((T, hq, D)).astype(np.float16)
    qkv = torch.from_numpy(np.concatenate([q, k, v], axis=1)).cuda()
    ws = w4.Kv4Workspace(batch, hq, cache)
    w4.kv4_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cache, batch, ws)
    y = w4.kv4_attention(qkv[:, :hq], cache, batch, ws)
    few = w4.Kv4Batch(batch.page_table, batch.lengths, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), 2, 1)
    one = w4.kv4_attention(qkv[[89, 122]][:, :hq], cache, few, ws)
    assert w4.device_status(ws) == 0
    kv, vv = split(kv_ref.values(k), lens), split(kv_ref.values(v), lens)
    for b, (qq, yy) in enumerate(zip(split(q, nq), split(y.cpu().numpy(), nq))):
        ref = kv_ref.attention(qq, kv[b], vv[b], nq[b], D ** -0.5)
        close(yy, ref, vv[b])
        close(one[b:b + 1].cpu().numpy(), ref[-1:], vv[b])


def test_refusals():
    import w4a16_mixed_precision_gb300 as w4
    k, v, cache, batch, hist = make([40], [1], 2, 128, 16, seed=14)
    ws = w4.Kv4Workspace(batch, 4, cache)
    q = torch.zeros((1, 4, 128), dtype=torch.float16, device="cuda")
    for bad in (q.float(), q.cpu(), q[:, :, :64], q.expand(2, 4, 128), q.transpose(1, 2)):
        with pytest.raises(ValueError):
            w4.kv4_attention(bad, cache, batch, ws)
    with pytest.raises(ValueError):
        w4.kv4_append(q[:, :2], q[:, :3], cache, batch, ws)
    for n in (3, 1):   # 3 query heads on 2 key heads; fewer query heads than key heads
        with pytest.raises(w4.MarlinError) as e:
            w4.kv4_attention(torch.zeros((1, n, 128), dtype=torch.float16, device="cuda"), cache, batch, ws)
        assert e.value.status == 1
    with pytest.raises(w4.MarlinError):
        w4.kv4_attention(q, cache, batch, ws, window=-1)
    with pytest.raises(w4.MarlinError):
        w4.kv4_attention(q, cache, batch, ws, scale=float("nan"))
    for args, status in (((4, 2, 96, 16), 2), ((4, 2, 128, 24), 2), ((0, 2, 128, 16), 1), ((4, 2, 128, 2048), 2)):
        with pytest.raises(w4.MarlinError) as e:
            w4.Kv4Cache(*args)
        assert e.value.status == status
    with pytest.raises(ValueError):
        w4.Kv4Batch(batch.page_table.long(), batch.lengths, batch.q_start, 1, 1)
    with pytest.raises(ValueError):
        w4.Kv4Batch(batch.page_table, batch.lengths, batch.lengths, 1, 1)
    odd = torch.zeros((1, 4 * 128 + 4), dtype=torch.float16, device="cuda")[:, 4:].view(1, 4, 128)
    with pytest.raises(w4.MarlinError) as e:
        w4.kv4_attention(odd, cache, batch, ws)
    assert e.value.status == 3
    # no tokens: nothing to do
    none = w4.Kv4Batch(batch.page_table, batch.lengths, torch.zeros_like(batch.q_start), 0, 0)
    assert w4.kv4_attention(q[:0], cache, none, ws).shape == (0, 4, 128)
    assert w4.device_status(ws) == 0
