"""Measured cases of the operators that verify trees of drafted tokens over the 4-bit cache.

A step that verifies drafted trees makes, for each request's new tokens (a tree, each with its parent):

  tree       from the parents: which new tokens each one sees (bits), and its position;
  rope       queries and keys are rotated by their positions (on one axis or several), the rotated keys
             and the values are quantised to 4 bits and written into the paged cache (read back: `kv4_read`);
  attention  softmax(q . K^T * scale) . V over that cache: every cached token before the new ones, and
             of the new ones those whose bit is set;
  compact    the kept tokens' entries move together, in the caches of all layers (read back again);
  copy       whole pages are copied, in the caches of all layers, when a request forks.

`listed` and `draw` give the cases, `prepare` what a program has in hand before the call, `run` one
pass, `work` the bytes and operations it cannot do without, `exact` the same outputs in 64 bits.
With `own` false `run` computes in elementary torch operations in 32 bits; with it true it calls this
repository's operators.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one request's 64 drafted tokens: latency
        dict(name="tree-one", op="tree", B=1, nq=64, ragged_q=False, L=900),
        # a batch of requests with trees of different sizes
        dict(name="tree-batch", op="tree", B=200, nq=157, ragged_q=True, L=5000),
        # a tree of 13 for each of 16 requests (70B: 64 query heads on 8), far positions of one axis
        dict(name="rope-trees", op="rope", B=16, nq=13, ragged_q=False, L=100000, Hq=64, Hkv=8, D=128, page=64, rot=128,
             axes=1, pairing="halves"),
        # prompts of 6 requests with images in them: time, height and width, 7B-like heads
        dict(name="rope-prompts-images", op="rope", B=6, nq=2300, ragged_q=True, L=2300, Hq=32, Hkv=8, D=128, page=16,
             rot=128, axes=3, pairing="halves"),
        # one request, a tree of 8, one key head for each query head (7B): latency
        dict(name="attention-one-tree", op="attention", B=1, nq=8, ragged_q=False, L=700, Hq=32, Hkv=32, D=128, page=64,
             window=0),
        # a batch of trees of up to 60, grouped heads (70B)
        dict(name="attention-trees", op="attention", B=14, nq=60, ragged_q=True, L=6000, Hq=64, Hkv=8, D=128, page=64,
             window=0),
        # one request with a long context and a tree of 25
        dict(name="attention-long", op="attention", B=1, nq=25, ragged_q=False, L=100001, Hq=64, Hkv=8, D=128, page=128,
             window=0),
        # small trees, heads of 64 channels, a sliding window, small pages
        dict(name="attention-window", op="attention", B=24, nq=5, ragged_q=False, L=6001, Hq=24, Hkv=8, D=64, page=16,
             window=2048),
        # the accepted path of each of 40 requests' trees of 61, in all 32 layers
        dict(name="compact-accepted", op="compact", B=40, nq=61, ragged_q=False, L=260, Hkv=8, D=128, page=64, layers=32,
             kept="path"),
        # dropping half of two long contexts' tokens, into new pages
        dict(name="compact-evict", op="compact", B=2, nq=50001, ragged_q=True, L=50001, Hkv=8, D=128, page=64, layers=1,
             kept="half"),
        # one request forks: its last page in all 32 layers
        dict(name="copy-fork-one", op="copy", pairs=1, n_pages=16, Hkv=8, D=128, page=64, layers=32),
        # a beam's 45 last pages in all 32 layers
        dict(name="copy-fork-beams", op="copy", pairs=45, n_pages=100, Hkv=8, D=128, page=64, layers=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "rope", "rope", "attention", "attention", "attention", "attention", "compact", "copy"])
    if op == "tree":
        nq = _log(rng, 1, 157)
        return dict(op=op, B=_log(rng, 1, 200), nq=nq, ragged_q=rng.random() < 0.5, L=nq + _log(rng, 1, 100000))
    page, D = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    if op == "copy":
        layers = rng.choice([1, 8, 32, 48])
        pairs = max(1, min(_log(rng, 1, 2000), 4000 // (layers * page // 16)))
        return dict(op=op, pairs=pairs, n_pages=2 * pairs + rng.randint(1, 9), Hkv=rng.choice([4, 8]), D=D, page=page,
                    layers=layers)
    if op == "rope":
        nq = _log(rng, 1, 2300)
        Hkv, G = rng.choice([(8, 8), (8, 4), (8, 3), (4, 7), (32, 1)])
        B = max(1, min(_log(rng, 1, 64), 100000000 // (nq * Hkv * (2 * G + 4) * D)))
        return dict(op=op, B=B, nq=nq, ragged_q=nq > 8 and rng.random() < 0.5, L=nq + _log(rng, 1, 100000 // B), Hq=Hkv * G,
                    Hkv=Hkv, D=D, page=page, rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 1, 2, 3]),
                    pairing=rng.choice(["halves", "halves", "neighbours"]))
    if op == "compact":
        Hkv = rng.choice([4, 8])
        if rng.random() < 0.5:
            nq, layers = _log(rng, 2, 157), rng.choice([1, 8, 32])
            B = max(1, min(_log(rng, 1, 64), 3000 // nq, 60000 // (nq * layers)))
            return dict(op=op, B=B, nq=nq, ragged_q=nq > 8 and rng.random() < 0.5, L=nq + _log(rng, 1, 500), Hkv=Hkv, D=D,
                        page=page, layers=layers, kept="path")
        nq = _log(rng, 100, 38000)
        return dict(op=op, B=rng.choice([1, 2]), nq=nq, ragged_q=rng.random() < 0.5, L=nq, Hkv=Hkv, D=D, page=page, layers=1,
                    kept="half")
    Hkv, G = rng.choice([(8, 8), (8, 4), (8, 3), (32, 1), (4, 7), (2, 16)])
    nq = _log(rng, 1, 100)
    L = _log(rng, 64, min(60000, 140000000 // (nq * Hkv * G))) + nq
    B = max(1, min(_log(rng, 1, 24), 800000 // (L * Hkv), 100000000 // (L * nq * Hkv * G)))
    return dict(op=op, B=B, nq=nq, ragged_q=nq > 8 and rng.random() < 0.5, L=L, Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                window=rng.choice([0, 0, 0, 512, 4096]))


def _lengths(case):
    """(new tokens, cached length with them) of each request: different ones, the same for every seed."""
    nq, lens = [], []
    for b in range(case["B"]):
        part = 1.0 - 0.75 * ((b * 0.6180339887) % 1.0)
        n = max(1, int(case["nq"] * part)) if case["ragged_q"] else case["nq"]
        nq.append(n)
        lens.append(n + int((case["L"] - case["nq"]) * part))
    return nq, lens


def _parents(case):
    """Each new token's parent among its request's (-1: the last cached token), parents first: mostly one of
    the tokens shortly before, so that trees are some levels deep.  The same for every seed."""
    out = []
    for b, n in enumerate(_lengths(case)[0]):
        rng = random.Random(1000 * b + n)
        out.append([-1] + [max(0, i - 1 - int(rng.expovariate(1 / 5.0))) for i in range(1, n)])
    return out


def _ancestors(parents):
    """For each token the tokens on its path from the root, its own included."""
    paths = []
    for i, p in enumerate(parents):
        paths.append((paths[p] if p >= 0 else []) + [i])
    return paths


def _kept(case):
    """The new tokens that each request keeps, ascending: the root and four others of a tree, or half of all."""
    out = []
    for b, n in enumerate(_lengths(case)[0]):
        rng = random.Random(77 * b + n)
        if case["kept"] == "half":
            out.append([i for i in range(n) if rng.random() < 0.5] or [0])
        else:
            k = min(4, max(0, n - 5))
            out.append([0] + sorted(rng.sample(range(5, n), k)))
    return out


def work(case):
    op = case["op"]
    if op == "copy":
        per = case["Hkv"] * case["page"] * 2 * (case["D"] // 2 + 4)
        return {"bytes": 2 * case["pairs"] * case["layers"] * per, "flops": 0}
    nq, lens = _lengths(case)
    T = sum(nq)
    if op == "tree":
        return {"bytes": T * 4 * (1 + -(-max(nq) // 32) + 1), "flops": 0}
    Hkv, D = case["Hkv"], case["D"]
    entry = Hkv * 2 * (D // 2 + 4)  # of a token in the cache
    if op == "compact":  # moved, then read and written as 16-bit values
        kept = sum(len(k) for k in _kept(case))
        return {"bytes": kept * case["layers"] * (3 * entry + Hkv * 2 * D * 2), "flops": 0}
    if op == "rope":  # vectors in, queries and cache entries out, entries read again and written as 16-bit values
        table = len(set(_flat_positions(case))) * case["rot"] * 4
        return {"bytes": T * ((2 * case["Hq"] + 4 * Hkv) * D * 2 + 2 * entry) + table, "flops": 3 * T * (case["Hq"] + Hkv) * case["rot"]}
    window, cached, pairs = case["window"], 0, 0
    for n, length, parents in zip(nq, lens, _parents(case)):
        first = length - n
        depth = [len(p) for p in _ancestors(parents)]
        seen = [first if not window else max(0, min(first, window - d)) for d in depth]
        cached += n + max(seen)
        pairs += sum(seen) + sum(depth)
    return {"bytes": cached * entry + 2 * T * case["Hq"] * D * 2, "flops": 4 * pairs * case["Hq"] * D}


# ---- the inputs ----------------------------------------------------------------------------

def _flat_positions(case):
    """Rows of the table that the new tokens use, one for each token and axis, token by token: text in order, and in
    prompts with several axes images of 24 columns, whose patches share a time and differ in row and column."""
    out = []
    for n, length in zip(*_lengths(case)):
        at = length - n
        for i in range(n):
            if case["axes"] > 1 and i % 700 >= 100:  # an image of up to 600 patches after 100 tokens of text
                patch = i % 700 - 100
                start = at + i - patch
                out += [(start, start + patch // 24, start + patch % 24)[a] for a in range(case["axes"])]
            else:
                out += [at + i] * case["axes"]
    return out


def _table(case):
    """cos and sin of position * 10000^(-2 j / rot), fp32, for every position and pair."""
    n = max(_flat_positions(case)) + 1
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
    angle = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _axis_of_pair(case):
    """Sections of the pairs, the first (time) half as long as the others where there are three."""
    half, axes = case["rot"] // 2, case["axes"]
    ends = {1: [half], 2: [half // 2, half], 3: [half // 4, half // 4 + (half - half // 4) // 2, half]}[axes]
    return [next(a for a, end in enumerate(ends) if j < end) for j in range(half)]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tree_bits(case):
    """int32 [T, words]: bit j of a row is set where the token sees the j-th new token of its request."""
    words = -(-max(_lengths(case)[0]) // 32)
    rows = []
    for parents in _parents(case):
        for path in _ancestors(parents):
            bits = sum(1 << j for j in path)
            rows.append([(((bits >> (32 * w)) & 0xFFFFFFFF) ^ 0x80000000) - 0x80000000 for w in range(words)])
    return _i32(rows)


def _inputs(case, seed):
    """Keys with a few strong channels, as models have them, values and queries; pages of the cache dealt out
    in random order."""
    g = torch.Generator(DEV).manual_seed(seed)
    op = case["op"]
    if op == "copy":
        size = case["Hkv"] * case["page"] * 2 * (case["D"] // 2 + 4)
        order = torch.randperm(case["n_pages"], generator=g, device=DEV).to(torch.int32)
        return dict(pages=[torch.randint(0, 256, (case["n_pages"], size), generator=g, device=DEV, dtype=torch.uint8)
                           for _ in range(case["layers"])],
                    src=order[:case["pairs"]].contiguous(), dst=order[case["pairs"]:2 * case["pairs"]].contiguous())
    nq, lens = _lengths(case)
    B, T, H = case["B"], sum(nq), sum(lens)
    start = _i32([sum(nq[:b]) for b in range(B + 1)])
    if op == "tree":
        # the seed moves every request by some positions
        shift = torch.randint(0, 50, (B,), generator=g, device=DEV, dtype=torch.int32)
        return dict(parents=_i32([p for request in _parents(case) for p in request]), lens=_i32(lens) + shift, q_start=start)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    normal = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.float16)  # noqa: E731
    per = [-(-x // page) for x in lens]
    order = torch.randperm(2 * sum(per) + 3, generator=g, device=DEV).to(torch.int32)
    tables = torch.zeros((2, B, max(per)), dtype=torch.int32, device=DEV)
    at = 0
    for i in range(2):
        for b in range(B):
            tables[i, b, :per[b]] = order[at:at + per[b]]
            at += per[b]
    d = dict(n_pages=len(order), page_table=tables[0].contiguous(), lens=_i32(lens), q_start=start)
    bias = normal(Hkv, D) * (torch.rand((Hkv, D), generator=g, device=DEV) < 0.06) * 4
    if op == "rope":
        d["q"], d["k"], d["v"] = normal(T, case["Hq"] + 2 * Hkv, D).split([case["Hq"], Hkv, Hkv], dim=1)
        d["k"] += bias
        d["positions"] = _i32(_flat_positions(case)).view(T, case["axes"]).t().contiguous()
        return d
    if op == "compact":
        d["k"], d["v"] = (normal(case["layers"], T, Hkv, D) for _ in "kv")
        d["k"] += bias
        kept = _kept(case)
        d["kept"] = _i32([len(x) for x in kept])
        d["index"] = _i32([i for x, n in zip(kept, nq) for i in x + [0] * (n - len(x))])
        d["into"] = tables[1].contiguous() if case["kept"] == "half" else None
        return d
    d["h_start"] = _i32([sum(lens[:b]) for b in range(B + 1)])
    d["k"], d["v"], d["q"] = normal(H, Hkv, D) + bias, normal(H, Hkv, D), normal(T, case["Hq"], D)
    d["tree"] = _tree_bits(case)
    return d


def _slots(table, lens, start, T, page):
    """The place in the cache of the last tokens of each request, token by token."""
    t = torch.arange(T, device=DEV)
    b = torch.bucketize(t, start[1:].long(), right=True)
    pos = lens.long()[b] - start.long()[b + 1] + t
    return table.long()[b, pos // page] * page + pos % page


def _quantise(x):
    """Codes 0..15, and the scale and offset (16 bits each) of every vector: a code c stands for
    s * (c - 8) + o, with s = (max - min) / 15 and o = min + 8 s."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).half()
    o = (lo + 8 * s.float()).half()
    c = torch.where(s > 0, torch.round((x - o.float()) / s.float()), torch.zeros((), device=x.device))
    return (c.clamp(-8, 7) + 8).to(torch.uint8), s, o


def _new_cache(n_pages, case):
    n, Hkv, D = n_pages * case["page"], case["Hkv"], case["D"]
    new = lambda *s, **k: torch.zeros(s, device=DEV, **k)  # noqa: E731
    return {x + y: new(n, Hkv, D, dtype=torch.uint8) if y == "c" else new(n, Hkv, 1, dtype=torch.float16)
            for x in "kv" for y in "cso"}


def _store(cache, k, v, at):
    for x, t in (("k", k), ("v", v)):
        cache[x + "c"][at], cache[x + "s"][at], cache[x + "o"][at] = _quantise(t)


def _load(cache, x, at):
    return (cache[x + "c"][at].float() - 8) * cache[x + "s"][at].float() + cache[x + "o"][at].float()


def _kept_batch(case, d):
    """A batch that reads the kept tokens back: of every layer in turn, in one cache that holds all layers."""
    layers, n_pages = case["layers"], d["n_pages"]
    nq, lens = _lengths(case)
    kept = [len(x) for x in _kept(case)]
    table = d["page_table"] if d["into"] is None else d["into"]
    tables = torch.cat([table + n_pages * i for i in range(layers)])
    ends = [length - n + k for length, n, k in zip(lens, nq, kept)] * layers
    counts = kept * layers
    start = [0]
    for k in counts:
        start.append(start[-1] + k)
    return tables.contiguous(), _i32(ends), _i32(start), start[-1], max(counts)


def prepare(case, seed):
    op = case["op"]
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import w4a16_mixed_precision_gb300 as w4
    if op == "copy":
        if own:
            st["caches"] = [w4.Kv4Cache(case["n_pages"], case["Hkv"], case["D"], case["page"]) for _ in range(case["layers"])]
            for cache, pages in zip(st["caches"], st["pages"]):
                cache.buf.copy_(pages.view(-1))
            batch = w4.Kv4Batch(_i32([[0]]), _i32([0]), _i32([0, 0]), 0, 0)
            st["ws"] = w4.Kv4Workspace(batch, case["Hkv"], st["caches"][0])
            st["pages"] = [c.buf.view(case["n_pages"], -1) for c in st["caches"]]
        return st
    nq, lens = _lengths(case)
    if op == "tree":
        if own:
            st["batch"] = w4.Kv4Batch(torch.zeros((case["B"], 1), dtype=torch.int32, device=DEV), st["lens"], st["q_start"],
                                      sum(nq), max(nq))
            st["ws"] = w4.Kv4Workspace(st["batch"], 1, w4.Kv4Cache(1, 1, 64, 16))
        return st
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if op == "rope":
        st["cos"], st["sin"] = _table(case)
    if own:
        layers = case.get("layers", 1)
        st["cache"] = w4.Kv4Cache(st["n_pages"] * layers, Hkv, D, page)
        st["batch"] = w4.Kv4Batch(st["page_table"], st["lens"], st["q_start"], sum(nq), max(nq))
        st["ws"] = w4.Kv4Workspace(st["batch"], case.get("Hq", Hkv), st["cache"])
        if op == "rope":
            st["rope"] = w4.Kv4Rope(st["cos"], st["sin"], axes=_axis_of_pair(case),
                                    interleaved=case["pairing"] == "neighbours")
        if op == "attention":
            w4.kv4_append(st["k"], st["v"], st["cache"],
                          w4.Kv4Batch(st["page_table"], st["lens"], st["h_start"], sum(lens), max(lens)), st["ws"])
        if op == "compact":  # the layers' caches lie one after the other, to be read back together
            st["layers"] = []
            for i, part in enumerate(st["cache"].buf.chunk(layers)):
                st["layers"].append(w4.Kv4Cache(1, Hkv, D, page))
                st["layers"][i].buf, st["layers"][i].n_pages = part, st["n_pages"]
                w4.kv4_append(st["k"][i], st["v"][i], st["layers"][i], st["batch"], st["ws"])
            st["kept_batch"] = w4.Kv4Batch(*_kept_batch(case, st))
    else:
        if op == "compact":
            st["layers"] = [_new_cache(st["n_pages"], case) for _ in range(case["layers"])]
            at = _slots(st["page_table"], st["lens"], st["q_start"], sum(nq), page)
            for i, cache in enumerate(st["layers"]):
                _store(cache, st["k"][i], st["v"][i], at)
        else:
            st["cache"] = _new_cache(st["n_pages"], case)
        if op == "attention":
            _store(st["cache"], st["k"], st["v"], _slots(st["page_table"], st["lens"], st["h_start"], sum(lens), page))
    if op != "rope":
        del st["k"], st["v"]
    return st


# ---- one pass ------------------------------------------------------------------------------

def _plain_tree(st, case):
    """The ancestors' bits by doubling: after step s a row holds its next 2^s ancestors."""
    start, parents = st["q_start"].long(), st["parents"].long()
    T, B, words = parents.shape[0], case["B"], -(-max(_lengths(case)[0]) // 32)
    t = torch.arange(T, device=DEV)
    b = torch.bucketize(t, start[1:], right=True)
    j = t - start[b]
    up = torch.where(parents < 0, T, start[b] + parents)  # the row of the parent, T for none
    up = torch.cat([up, up.new_full((1,), T)])
    word = torch.arange(words, device=DEV)
    bits = torch.where(word == (j // 32)[:, None], (1 << (j % 32))[:, None], 0)
    bits = torch.cat([bits, bits.new_zeros((1, words))])
    depth = torch.cat([torch.ones_like(t), t.new_zeros(1)])
    steps = max(1, max(_lengths(case)[0]).bit_length())
    for _ in range(steps):
        bits, depth, up = bits | bits[up], depth + depth[up], up[up]
    mask = torch.where(bits >= 2**31, bits - 2**32, bits)[:T].to(torch.int32)
    first = st["lens"].long() - (start[1:] - start[:-1])
    return mask, (first[b] + depth[:T] - 1).to(torch.int32)


def _rotated(x, c, s, case):
    """The pairs (x1, x2) of the first `rot` channels become (x1 c - x2 s, x2 c + x1 s)."""
    rot, x = case["rot"], x.float()
    if case["pairing"] == "halves":
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    else:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).half()


def _plain_rope(st, case):
    pair = torch.arange(case["rot"] // 2, device=DEV)
    at = st["positions"].long()[torch.tensor(_axis_of_pair(case), device=DEV)].t()   # [T, pairs]
    c, s = st["cos"][at, pair][:, None], st["sin"][at, pair][:, None]
    q, k = _rotated(st["q"], c, s, case), _rotated(st["k"], c, s, case)
    slots = _slots(st["page_table"], st["lens"], st["q_start"], k.shape[0], case["page"])
    _store(st["cache"], k, st["v"], slots)
    return q, _load(st["cache"], "k", slots).half(), _load(st["cache"], "v", slots).half()


def _plain_attention(st, case):
    B, Hkv, D, page, window = case["B"], case["Hkv"], case["D"], case["page"], case["window"]
    G, L = case["Hq"] // Hkv, int(st["page_table"].shape[1]) * page
    nq, lens, T = max(_lengths(case)[0]), st["lens"].long(), st["q"].shape[0]
    j = torch.arange(L, device=DEV)
    at = st["page_table"].long()[:, j // page] * page + j % page                 # [B, L]
    k, v = (_load(st["cache"], x, at).permute(0, 2, 1, 3) for x in "kv")         # [B, Hkv, L, D]
    first, count = st["q_start"].long()[:-1], st["q_start"].long()[1:] - st["q_start"].long()[:-1]
    i = torch.arange(nq, device=DEV)
    rows = (first[:, None] + i).clamp(max=T - 1)                                 # [B, nq]
    q = st["q"].float()[rows].view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D)
    s = (q @ k.transpose(2, 3)).view(B, Hkv, G, nq, L) * (1.0 / math.sqrt(D))
    bits = (st["tree"][rows][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    bits = bits.flatten(2).bool()                                                # [B, nq, new]
    before = lens - count                                                        # cached tokens before the new ones
    new = j - before[:, None]                                                    # [B, L]
    see = (new < 0)[:, None, :].expand(B, nq, L)
    if window:  # of those before, by the row's depth in the tree
        see = see & (j > (before[:, None] + bits.sum(-1) - 1)[..., None] - window)
    mine = torch.gather(bits, 2, new.clamp(0, bits.shape[2] - 1)[:, None, :].expand(B, nq, L))
    see = see | (mine & ((new >= 0) & (new < count[:, None]))[:, None, :])
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (s - top).exp_()
    o = (p.view(B, Hkv, G * nq, L) @ v).view(B, Hkv, G, nq, D) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nq, case["Hq"], D)
    return o[i < count[:, None]].half()


def _plain_compact(st, case):
    T, page, start = st["index"].shape[0], case["page"], st["q_start"].long()
    t = torch.arange(T, device=DEV)
    b = torch.bucketize(t, start[1:], right=True)
    i, first = t - start[b], st["lens"].long()[b] - (start[b + 1] - start[b])
    live = i < st["kept"].long()[b]
    b, to, of = b[live], (first + i)[live], (first + st["index"].long())[live]
    into = st["page_table"] if st["into"] is None else st["into"]
    src = st["page_table"].long()[b, of // page] * page + of % page
    dst = into.long()[b, to // page] * page + to % page
    ks, vs = [], []
    for cache in st["layers"]:
        for name in cache:
            cache[name][dst] = cache[name][src]
        ks.append(_load(cache, "k", dst).half())
        vs.append(_load(cache, "v", dst).half())
    new = st["lens"] - (st["q_start"][1:] - st["q_start"][:-1]) + st["kept"]
    return new, torch.cat(ks), torch.cat(vs)


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import w4a16_mixed_precision_gb300 as w4
        if op == "tree":
            return w4.kv4_tree(state["parents"], state["batch"], state["ws"])
        if op == "rope":
            q = w4.kv4_rope_append(state["q"], state["k"], state["v"], state["positions"], state["rope"], state["cache"],
                                   state["batch"], state["ws"])
            return (q, *w4.kv4_read(state["cache"], state["batch"], state["ws"]))
        if op == "attention":
            return w4.kv4_tree_attention(state["q"], state["cache"], state["batch"], state["tree"], state["ws"],
                                         window=case["window"])
        if op == "compact":
            lengths = w4.kv4_compact(state["layers"], state["batch"], state["index"], state["kept"], state["ws"],
                                     into=state["into"])
            return (lengths, *w4.kv4_read(state["cache"], state["kept_batch"], state["ws"]))
        w4.kv4_copy_pages(state["caches"], state["src"], state["dst"], state["ws"])
        return state["pages"]
    if op == "tree":
        return _plain_tree(state, case)
    if op == "rope":
        return _plain_rope(state, case)
    if op == "attention":
        return _plain_attention(state, case)
    if op == "compact":
        return _plain_compact(state, case)
    src, dst = state["src"].long(), state["dst"].long()
    for pages in state["pages"]:
        pages[dst] = pages[src]
    return state["pages"]


# ---- the same in 64 bits -------------------------------------------------------------------

def _exact_values(x):
    """What the cache holds for the vectors x: by the format, scale and offset are rounded to 16 bits."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).float().half().double()
    o = (lo + 8 * s).half().double()
    code = torch.minimum(torch.maximum(((x - o) / s).round(), torch.full_like(x, -8)), torch.full_like(x, 7))
    return torch.where(s > 0, o + s * code, o)


def _exact_rope(case, d):
    cos, sin = (t.double() for t in _table(case))
    axis, rot, half = _axis_of_pair(case), case["rot"], case["rot"] // 2
    out = []
    for x in (d["q"].double(), d["k"].double()):
        y = x.clone()
        for j in range(half):
            at = d["positions"][axis[j]].long()
            c, s = cos[at, j][:, None], sin[at, j][:, None]
            a, b = (j, j + half) if case["pairing"] == "halves" else (2 * j, 2 * j + 1)
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        out.append(y)
    # the cache quantises the rotated keys as 16-bit numbers
    return out[0], _exact_values(out[1].half()), _exact_values(d["v"])


def _exact_attention(case, d):
    k, v = _exact_values(d["k"]), _exact_values(d["v"])
    nq, lens = _lengths(case)
    G, out = case["Hq"] // case["Hkv"], torch.empty(d["q"].shape, dtype=torch.float64, device=DEV)
    t = h = 0
    for n, length, parents in zip(nq, lens, _parents(case)):
        first = length - n
        hide = torch.ones((n, length), dtype=torch.bool)
        for i, path in enumerate(_ancestors(parents)):
            lo = max(0, first + len(path) - case["window"]) if case["window"] else 0
            hide[i, lo:first] = False
            hide[i, [first + j for j in path]] = False
        hide = hide.to(DEV)
        for head in range(case["Hq"]):
            s = d["q"][t:t + n, head].double() @ k[h:h + length, head // G].t() / math.sqrt(case["D"])
            p = torch.softmax(s.masked_fill(hide, -math.inf), dim=-1)
            out[t:t + n, head] = p @ v[h:h + length, head // G]
        t, h = t + n, h + length
    return out


def exact(case, seed):
    d, op = _inputs(case, seed), case["op"]
    if op == "tree":
        depth = [len(path) for parents in _parents(case) for path in _ancestors(parents)]
        counts = torch.tensor(_lengths(case)[0], device=DEV)
        first = torch.repeat_interleave(d["lens"].long() - counts, counts)
        return _tree_bits(case), (first + torch.tensor(depth, device=DEV) - 1).to(torch.int32)
    if op == "copy":
        for pages in d["pages"]:
            for a, b in zip(d["src"].tolist(), d["dst"].tolist()):
                pages[b] = pages[a]
        return d["pages"]
    if op == "rope":
        return _exact_rope(case, d)
    if op == "attention":
        return _exact_attention(case, d)
    nq, lens = _lengths(case)
    rows, t = [], 0
    for n, kept in zip(nq, _kept(case)):
        rows += [t + i for i in kept]
        t += n
    rows = torch.tensor(rows, device=DEV)
    new = [length - n + len(x) for n, length, x in zip(nq, lens, _kept(case))]
    return _i32(new), *(torch.cat([_exact_values(x[rows]) for x in d[name]]) for name in "kv")
