"""Measured cases of the operators around the W4A16 products of a served model.

Three operators of one attention block, for many requests at once:

  lora        y = x . dequant(W) + scaling[a] * (x . A[a]^T) . B[a]^T, row by row, where a is the
              low-rank adapter of the row's request (or none) beside the shared 4-bit projection;
  append      new keys and values are quantised to 4 bits and written into a paged cache (the cached
              values are read back: `kv4_read`);
  attention   softmax(q . K^T * scale) . V over that cache, causal, for single tokens and for prompts.

`listed` and `draw` give the cases, `prepare` what a program has in hand before the call, `run` one
pass, `work` the bytes and operations it cannot do without, `exact` the same outputs in 64 bits.
With `own` false `run` computes in elementary torch operations in 32 bits; with it true it calls this
repository's operators.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ---- the cases -----------------------------------------------------------------------------

def listed():
    return [
        # one token of one request through a 4096 x 4096 projection with a rank-16 adapter: latency
        dict(name="lora-one-token", op="lora", M=1, K=4096, N=4096, group=128, zeros=False, r=16,
             adapters=8, share=1),
        # a decode batch on the 7B QKV projection; every request has its own adapter or none
        dict(name="lora-decode-32", op="lora", M=32, K=4096, N=12288, group=128, zeros=False, r=16,
             adapters=24, share=1),
        # odd batch, explicit zeros, one scale per column, few adapters of a higher rank shared by many rows
        dict(name="lora-decode-45-zeros", op="lora", M=45, K=8192, N=10240, group=8192, zeros=True, r=64,
             adapters=5, share=3),
        # prompts of several requests: long runs of rows with the same adapter
        dict(name="lora-prompts", op="lora", M=1990, K=4096, N=12288, group=128, zeros=False, r=32,
             adapters=6, share=331),
        # one new token for each of 48 requests into the cache: latency
        dict(name="append-decode-48", op="append", B=48, nq=1, ragged_q=False, L=1777, Hkv=8, D=128, page=64),
        # the prompts of 6 requests of different lengths
        dict(name="append-prompts", op="append", B=6, nq=2500, ragged_q=True, L=2500, Hkv=8, D=128, page=16),
        # one request, one token, 32 key and value heads (7B): latency
        dict(name="attention-one-token", op="attention", B=1, nq=1, ragged_q=False, L=700, Hq=32, Hkv=32, D=128,
             page=64, window=0),
        # a decode batch with grouped heads (70B: 64 query heads on 8), requests of different lengths
        dict(name="attention-decode-40", op="attention", B=40, nq=1, ragged_q=False, L=7900, Hq=64, Hkv=8, D=128,
             page=64, window=0),
        # one request with a very long context: the work of each head is split over the whole card
        dict(name="attention-long", op="attention", B=1, nq=1, ragged_q=False, L=131001, Hq=64, Hkv=8, D=128,
             page=128, window=0),
        # verifying 5 proposed tokens each, heads of 64 channels, a sliding window, small pages
        dict(name="attention-verify-window", op="attention", B=16, nq=5, ragged_q=False, L=6001, Hq=24, Hkv=8, D=64,
             page=16, window=2048),
        # the next 1000 tokens of a long prompt against what is cached of it
        dict(name="attention-chunk", op="attention", B=1, nq=1000, ragged_q=False, L=9000, Hq=64, Hkv=8, D=128,
             page=64, window=0),
        # the whole prompts of 5 requests of different lengths, one key head for each query head (7B)
        dict(name="attention-prompts", op="attention", B=5, nq=1900, ragged_q=True, L=1900, Hq=32, Hkv=32, D=128,
             page=32, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "append", "attention", "attention", "attention", "attention"])
    if op == "lora":
        K, N = rng.choice([(4096, 12288), (4096, 4096), (11008, 4096), (8192, 10240), (8192, 8192), (2048, 5632),
                           (13824, 5120)])
        M = _log(rng, 1, 2000)
        return dict(op=op, M=M, K=K, N=N, group=rng.choice([128, 128, K]), zeros=rng.random() < 0.4,
                    r=rng.choice([8, 16, 32, 64]), adapters=rng.randint(1, 24),
                    share=1 if M < 64 else rng.randint(M // 8, M // 2))
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        nq = _log(rng, 1, 2500)
        B = max(1, min(64, 15000 // nq, _log(rng, 1, 64)))
        return dict(op=op, B=B, nq=nq, ragged_q=nq > 8 and rng.random() < 0.5, L=nq + _log(rng, 1, 2000),
                    Hkv=rng.choice([4, 8, 32]) if nq * B < 4000 else 8, D=rng.choice([64, 128]), page=page)
    Hkv, G = rng.choice([(8, 8), (8, 4), (8, 3), (32, 1), (4, 7), (2, 16)])
    form = rng.choice(["decode", "decode", "verify", "prompt"])
    if form == "prompt":
        nq = _log(rng, 64, 1500)
        B = max(1, min(5, 1500 // nq))
        L = nq + (_log(rng, 1, 6000) if rng.random() < 0.5 else 0)
    else:
        nq = 1 if form == "decode" else rng.randint(2, 8)
        L = _log(rng, 64, 100000) + nq
        B = max(1, min(_log(rng, 1, 64), 2000000 // (L * Hkv)))
    return dict(op=op, B=B, nq=nq, ragged_q=form == "prompt" and rng.random() < 0.5, L=L, Hq=Hkv * G, Hkv=Hkv,
                D=rng.choice([64, 128, 128]), page=page, window=rng.choice([0, 0, 0, 512, 4096]))


def _lengths(case):
    """(query tokens, cached length with them) of each request: different ones, the same for every seed."""
    nq, lens = [], []
    for b in range(case["B"]):
        part = 1.0 - 0.75 * ((b * 0.6180339887) % 1.0)
        n = max(1, int(case["nq"] * part)) if case["ragged_q"] else case["nq"]
        nq.append(n)
        lens.append(n + int((case["L"] - case["nq"]) * part))
    return nq, lens


def _pairs(n, length, window):
    """Pairs of a query and a key that it sees, for the last n of `length` positions."""
    first = length - n
    if not window:
        return n * first + n * (n + 1) // 2
    return sum(min(window, first + i + 1) for i in range(n))


def _reach(n, length, window):
    """Cached positions that some of the last n queries see."""
    return length if not window else min(length, n + window - 1)


def work(case):
    if case["op"] == "lora":
        M, K, N, r = case["M"], case["K"], case["N"], case["r"]
        groups = K // case["group"]
        used = len(set(a for a in _adapter_of_row(case) if a >= 0))
        rows = sum(1 for a in _adapter_of_row(case) if a >= 0)
        weights = K * N // 2 + groups * N * 2 + (groups * N // 2 if case["zeros"] else 0)
        return {"bytes": weights + used * r * (K + N) * 2 + 2 * M * (K + N),
                "flops": 2 * M * K * N + 2 * rows * r * (K + N)}
    nq, lens = _lengths(case)
    T, Hkv, D = sum(nq), case["Hkv"], case["D"]
    if case["op"] == "append":  # the vectors in, 4-bit codes and two 16-bit numbers a vector out, and both ways again
        cached = T * Hkv * 2 * (D // 2 + 4)
        return {"bytes": 2 * (T * Hkv * 2 * D * 2 + cached), "flops": 0}
    window = case["window"]
    cached = sum(_reach(n, x, window) for n, x in zip(nq, lens)) * Hkv * 2 * (D // 2 + 4)
    pairs = sum(_pairs(n, x, window) for n, x in zip(nq, lens))
    return {"bytes": cached + 2 * T * case["Hq"] * D * 2, "flops": 4 * pairs * case["Hq"] * D}


# ---- the inputs ----------------------------------------------------------------------------

def _adapter_of_row(case):
    """The adapter of each row: runs of `share` rows, one run in eight without an adapter."""
    out = []
    for m in range(case["M"]):
        k = m // case["share"]
        out.append(-1 if k % 8 == 7 else (k * 5 + 1) % case["adapters"])
    return out


def _lora_inputs(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    M, K, N, r, n = case["M"], case["K"], case["N"], case["r"], case["adapters"]
    groups = K // case["group"]
    words = lambda *s: torch.randint(-2**31, 2**31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
    normal = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    return dict(
        x=normal(M, K).half(), q=words(K // 8, N),
        s=(0.02 * (0.5 + torch.rand((groups, N), generator=g, device=DEV))).half(),
        z=words(groups, N // 8) if case["zeros"] else None,
        a=(normal(n, r, K) / math.sqrt(K)).half(), b=(normal(n, N, r) * 0.5).half(),
        scaling=0.5 + torch.rand((n,), generator=g, device=DEV), index=torch.tensor(_adapter_of_row(case), dtype=torch.int32, device=DEV))


def _kv_inputs(case, seed):
    """Keys with a few strong channels, as models have them, values and queries; the history of each
    request in pages of the cache that are dealt out in random order."""
    g = torch.Generator(DEV).manual_seed(seed)
    nq, lens = _lengths(case)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    normal = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.float16)  # noqa: E731
    per = [-(-x // page) for x in lens]
    n_pages = sum(per) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((B, max(per)), dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    bias = normal(Hkv, D) * (torch.rand((Hkv, D), generator=g, device=DEV) < 0.06) * 4
    T, H = sum(nq), sum(lens)
    d = dict(page_table=table, n_pages=n_pages,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             q_start=torch.tensor([sum(nq[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV))
    if case["op"] == "append":
        d["k"], d["v"] = normal(T, Hkv, D) + bias, normal(T, Hkv, D)
    else:
        d["h_start"] = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
        d["k"], d["v"] = normal(H, Hkv, D) + bias, normal(H, Hkv, D)
        d["q"] = normal(T, case["Hq"], D)
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


def prepare(case, seed):
    if case["op"] == "lora":
        st = _lora_inputs(case, seed)
        if own:
            import w4a16_mixed_precision_gb300 as w4
            st["pw"] = w4.repack(st["q"], st["s"], st["z"], case["group"])
            st["bank"] = w4.LoraBank(st["a"], st["b"], st["scaling"])
            st["ws"] = w4.LoraWorkspace(case["M"], case["K"], case["N"], case["group"], case["r"])
        st["case"] = case
        return st
    st = _kv_inputs(case, seed)
    nq, lens = _lengths(case)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if own:
        import w4a16_mixed_precision_gb300 as w4
        st["cache"] = w4.Kv4Cache(st["n_pages"], Hkv, D, page)
        st["batch"] = w4.Kv4Batch(st["page_table"], st["lens"], st["q_start"], sum(nq), max(nq))
        st["ws"] = w4.Kv4Workspace(st["batch"], case.get("Hq", Hkv), st["cache"])
        if case["op"] == "attention":
            w4.kv4_append(st["k"], st["v"], st["cache"],
                          w4.Kv4Batch(st["page_table"], st["lens"], st["h_start"], sum(lens), max(lens)), st["ws"])
    else:
        n = st["n_pages"] * page
        new = lambda *s, **k: torch.zeros(s, device=DEV, **k)  # noqa: E731
        for x in "kv":
            st[x + "c"], st[x + "s"], st[x + "o"] = (new(n, Hkv, D, dtype=torch.uint8), new(n, Hkv, 1, dtype=torch.float16),
                                                     new(n, Hkv, 1, dtype=torch.float16))
        if case["op"] == "attention":
            _store(st, st["h_start"], sum(lens), page)
    if case["op"] == "attention":
        del st["k"], st["v"]
    st["case"] = case
    return st


# ---- one pass ------------------------------------------------------------------------------

def _store(st, start, T, page):
    at = _slots(st["page_table"], st["lens"], start, T, page)
    for x in "kv":
        st[x + "c"][at], st[x + "s"][at], st[x + "o"][at] = _quantise(st[x])


def _load(st, x, at):
    return (st[x + "c"][at].float() - 8) * st[x + "s"][at].float() + st[x + "o"][at].float()


def _unpack(words, dim):
    """int32 words of eight 4-bit codes -> the codes in 32-bit floats, eight times as many along `dim`."""
    shift = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    codes = (words.unsqueeze(dim + 1) >> shift.view(-1, *([1] * (words.dim() - dim - 1)))) & 15
    return codes.flatten(dim, dim + 1).float()


def _plain_lora(st, case):
    x, group, n, r = st["x"].float(), case["group"], case["adapters"], case["r"]
    z = _unpack(st["z"], 1).repeat_interleave(group, 0) if st["z"] is not None else 8.0
    # the weight that a code stands for is a 16-bit number by its definition
    w = ((_unpack(st["q"], 0) - z) * st["s"].float().repeat_interleave(group, 0)).half().float()
    mine = st["index"].long()[:, None] == torch.arange(n, device=x.device)
    v = (x @ st["a"].float().flatten(0, 1).t()).view(-1, n, r) * (mine * st["scaling"])[:, :, None]
    return (x @ w + v.flatten(1) @ st["b"].float().transpose(1, 2).flatten(0, 1)).half()


def _plain_attention(st, case):
    B, Hkv, D, page, window = case["B"], case["Hkv"], case["D"], case["page"], case["window"]
    G, L = case["Hq"] // Hkv, int(st["page_table"].shape[1]) * page
    nq, lens, T = max(_lengths(case)[0]), st["lens"].long(), st["q"].shape[0]
    j = torch.arange(L, device=DEV)
    at = st["page_table"].long()[:, j // page] * page + j % page                 # [B, L]
    k, v = (_load(st, x, at).permute(0, 2, 1, 3) for x in "kv")                  # [B, Hkv, L, D]
    first, count = st["q_start"].long()[:-1], st["q_start"].long()[1:] - st["q_start"].long()[:-1]
    i = torch.arange(nq, device=DEV)
    rows = (first[:, None] + i).clamp(max=T - 1)                                 # [B, nq]
    pos = (lens - count)[:, None] + i                                            # [B, nq]
    q = st["q"].float()[rows].view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D)
    s = (q @ k.transpose(2, 3)).view(B, Hkv, G, nq, L) * (1.0 / math.sqrt(D))
    see = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if window:
        see &= j > pos[:, :, None] - window
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (s - top).exp_()
    o = (p.view(B, Hkv, G * nq, L) @ v).view(B, Hkv, G, nq, D) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, nq, case["Hq"], D)
    return o[i < count[:, None]].half()


def run(state):
    case = state["case"]
    if own:
        import w4a16_mixed_precision_gb300 as w4
        if case["op"] == "lora":
            return w4.lora_gemm(state["x"], state["pw"], state["bank"], state["index"], state["ws"])
        if case["op"] == "append":
            w4.kv4_append(state["k"], state["v"], state["cache"], state["batch"], state["ws"])
            return w4.kv4_read(state["cache"], state["batch"], state["ws"])
        return w4.kv4_attention(state["q"], state["cache"], state["batch"], state["ws"], window=case["window"])
    if case["op"] == "lora":
        return _plain_lora(state, case)
    if case["op"] == "append":
        T = state["k"].shape[0]
        _store(state, state["q_start"], T, case["page"])
        at = _slots(state["page_table"], state["lens"], state["q_start"], T, case["page"])
        return _load(state, "k", at).half(), _load(state, "v", at).half()
    return _plain_attention(state, case)


# ---- the same in 64 bits -------------------------------------------------------------------

def _exact_values(x):
    """What the cache holds for the vectors x: by the format, scale and offset are rounded to 16 bits."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).float().half().double()
    o = (lo + 8 * s).half().double()
    code = torch.minimum(torch.maximum(((x - o) / s).round(), torch.full_like(x, -8)), torch.full_like(x, 7))
    return torch.where(s > 0, o + s * code, o)


def exact(case, seed):
    if case["op"] == "lora":
        d = _lora_inputs(case, seed)
        K, N, group = case["K"], case["N"], case["group"]
        w = torch.empty((K, N), dtype=torch.float64, device=DEV)
        for i in range(8):
            w[i::8] = ((d["q"] >> (4 * i)) & 15).double()
        for j in range(K // group):
            z = torch.full((N,), 8.0, dtype=torch.float64, device=DEV)
            if d["z"] is not None:
                for i in range(8):
                    z[i::8] = ((d["z"][j] >> (4 * i)) & 15).double()
            w[j * group:(j + 1) * group] = ((w[j * group:(j + 1) * group] - z) * d["s"][j].double()).half().double()
        x = d["x"].double()
        y = x @ w
        index = _adapter_of_row(case)
        for a in sorted(set(i for i in index if i >= 0)):
            rows = torch.tensor([m for m, i in enumerate(index) if i == a], device=DEV)
            y[rows] += float(d["scaling"][a]) * ((x[rows] @ d["a"][a].double().t()) @ d["b"][a].double().t())
        return y
    d = _kv_inputs(case, seed)
    k, v = _exact_values(d["k"]), _exact_values(d["v"])
    if case["op"] == "append":
        return k, v
    nq, lens = _lengths(case)
    G, out = case["Hq"] // case["Hkv"], torch.empty(d["q"].shape, dtype=torch.float64, device=DEV)
    t = h = 0
    for n, length in zip(nq, lens):
        key = torch.arange(length, device=DEV)
        pos = torch.arange(length - n, length, device=DEV)[:, None]
        hide = key > pos
        if case["window"]:
            hide = hide | (key + case["window"] <= pos)
        for head in range(case["Hq"]):
            s = d["q"][t:t + n, head].double() @ k[h:h + length, head // G].t() / math.sqrt(case["D"])
            p = torch.softmax(torch.where(hide, torch.full_like(s, -math.inf), s), dim=-1)
            out[t:t + n, head] = p @ v[h:h + length, head // G]
        t, h = t + n, h + length
    return out
