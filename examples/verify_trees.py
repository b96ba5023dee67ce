"""Speculative decoding over the 4-bit cache: each step a tree of drafted tokens for every request is run through the
model at once, the longest path that agrees with what the model itself would have said is kept, and its entries in the
caches of all layers move together.  A request can fork: the new one shares the pages that are full.  Random weights; the
drafts are guesses from a table of what followed a token before.

    python examples/verify_trees.py            # 4 requests, 24 steps
"""
from __future__ import annotations

import argparse
import os
import random
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import w4a16_mixed_precision_gb300 as w4


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """Layers of attention alone: 4-bit projections, rotary positions, a cache each."""

    def __init__(self, layers: int, hidden: int, heads: int, kv_heads: int, vocabulary: int, n_pages: int, page_size: int,
                 max_tokens: int, seed: int = 0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.d = heads, kv_heads, hidden // heads
        n_qkv = (heads + 2 * kv_heads) * self.d

        def projection(K, N):
            q = torch.randint(-2**31, 2**31, (K // 8, N), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
            s = ((0.5 + torch.rand((K // 128, N), generator=g, device="cuda")) * (0.25 / K ** 0.5)).half()
            return w4.repack(q, s, None, 128)

        self.layers = [(projection(hidden, n_qkv), projection(hidden, hidden)) for _ in range(layers)]
        self.caches = [w4.Kv4Cache(n_pages, kv_heads, self.d, page_size) for _ in range(layers)]
        self.words = torch.randn((vocabulary, hidden), generator=g, device="cuda").half()
        self.rope = w4.Kv4Rope.from_theta(self.d, 4096)
        self.qkv_ws, self.out_ws = (w4.Workspace(max_tokens, hidden, n, 128) for n in (n_qkv, hidden))
        self.kv_ws = w4.Kv4Workspace(w4.Kv4Batch(i32([[0]]), i32([0]), i32([0, max_tokens]), max_tokens, max_tokens), heads,
                                     self.caches[0])

    def __call__(self, tokens, batch: w4.Kv4Batch, parents):
        """The most likely next token after each of the batch's new tokens, trees with these parents."""
        mask, positions = w4.kv4_tree(parents, batch, self.kv_ws)
        x = self.words[tokens]
        for (qkv, out), cache in zip(self.layers, self.caches):
            y = w4.gemm(torch.nn.functional.rms_norm(x, x.shape[-1:]), qkv, self.qkv_ws).unflatten(1, (-1, self.d))
            q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
            q = w4.kv4_rope_append(q, k, v, positions, self.rope, cache, batch, self.kv_ws)
            o = w4.kv4_tree_attention(q, cache, batch, mask, self.kv_ws)
            x = x + w4.gemm(o.flatten(1), out, self.out_ws)
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.words.t()).argmax(-1)


class Request:
    def __init__(self, prompt):
        self.tokens = list(prompt)   # all of them; the last one is not in the caches yet
        self.pages, self.length = [], 0


class Server:
    def __init__(self, model: Model, pages: w4.Kv4Pages, max_pages: int, draft: int, seed: int = 0):
        self.model, self.pages, self.max_pages, self.draft = model, pages, max_pages, draft
        self.rng, self.followed, self.requests = random.Random(seed), {}, []

    def batch(self, new):
        """new[b] more tokens for request b, in pages of its own."""
        size = self.pages.page_size
        for r, n in zip(self.requests, new):
            r.pages += self.pages.take(max(0, -(-(r.length + n) // size) - len(r.pages)))
        table = torch.zeros((len(new), self.max_pages), dtype=torch.int32)
        for b, r in enumerate(self.requests):
            table[b, :len(r.pages)] = torch.tensor(r.pages, dtype=torch.int32)
        start = [sum(new[:b]) for b in range(len(new) + 1)]
        return w4.Kv4Batch(table.cuda(), i32([r.length + n for r, n in zip(self.requests, new)]), i32(start), start[-1], max(new))

    def admit(self, prompt):
        """A new request: its prompt but the last token is a tree without branches, of which all is kept.  (Prompts are short
        here: one of thousands of tokens is for kv4_attention, with its positions counted on.)"""
        self.requests.append(Request(prompt))
        new = [0] * (len(self.requests) - 1) + [len(prompt) - 1]
        self.model(torch.tensor(prompt[:-1], device="cuda"), self.batch(new), i32(range(-1, len(prompt) - 2)))
        self.requests[-1].length = len(prompt) - 1

    def fork(self, b: int):
        """Another request that goes on from what request b has, on its own."""
        old, new = self.requests[b], Request(self.requests[b].tokens)
        new.pages, copies = self.pages.fork(old.pages, old.length)
        new.length = old.length
        if copies:
            w4.kv4_copy_pages(self.model.caches, i32([a for a, _ in copies]), i32([c for _, c in copies]), self.model.kv_ws)
        self.requests.append(new)

    def tree(self, r: Request):
        """The request's last token and guesses of what follows it, two for every token."""
        tokens, parents = [r.tokens[-1]], [-1]
        at = 0
        while len(tokens) < self.draft and at < len(tokens):
            for guess in self.followed.get(tokens[at], [])[:2]:
                tokens.append(guess)
                parents.append(at)
            at += 1
        return tokens, parents

    def step(self):
        """One step of all requests; how many tokens each has got."""
        trees = [self.tree(r) for r in self.requests]
        batch = self.batch([len(t) for t, _ in trees])
        said = self.model(torch.tensor([t for tree, _ in trees for t in tree], device="cuda"), batch,
                          i32([p for _, parents in trees for p in parents])).tolist()
        index, kept, got, start = [], [], [], 0
        for r, (tokens, parents) in zip(self.requests, trees):
            path = [0]
            while True:  # the child that is what the model says after its parent
                want = said[start + path[-1]]
                known = self.followed.setdefault(tokens[path[-1]], [])
                if want not in known:
                    known.insert(0, want)
                child = next((c for c in range(len(tokens)) if parents[c] == path[-1] and tokens[c] == want), None)
                if child is None:
                    break
                path.append(child)
            r.tokens += [tokens[i] for i in path[1:]] + [said[start + path[-1]]]
            index += path + [0] * (len(tokens) - len(path))
            kept.append(len(path))
            got.append(len(path))
            start += len(tokens)
        lengths = w4.kv4_compact(self.model.caches, batch, i32(index), i32(kept), self.model.kv_ws).tolist()
        for r, n in zip(self.requests, lengths):
            r.length = n
            spare = -(-n // self.pages.page_size)
            self.pages.free(r.pages[spare:])
            del r.pages[spare:]
        return got


def serve(requests=4, steps=24, layers=3, hidden=1024, heads=8, kv_heads=2, vocabulary=50, draft=12, page_size=16, seed=0):
    """Requests with prompts of different lengths; after a third of the steps the first one forks.  Returns the server and
    the tokens that every step brought."""
    n_pages, max_pages = 64 * (requests + 1), 64
    model = Model(layers, hidden, heads, kv_heads, vocabulary, n_pages, page_size, (requests + 1) * max(draft, 64), seed)
    server = Server(model, w4.Kv4Pages(n_pages, page_size), max_pages, draft, seed)
    rng = random.Random(seed)
    for b in range(requests):
        server.admit([rng.randrange(vocabulary) for _ in range(5 + 13 * b)])
    got = []
    for i in range(steps):
        if i == steps // 3:
            server.fork(0)
        got.append(server.step())
    for name, ws in (("qkv", model.qkv_ws), ("out", model.out_ws), ("cache", model.kv_ws)):
        status = w4.device_status(ws)
        if status:
            raise RuntimeError(f"{name}: {w4.status_string(status)}")
    return server, got


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--draft", type=int, default=12)
    a = ap.parse_args()
    server, got = serve(a.requests, a.steps, draft=a.draft)
    tokens = sum(map(sum, got))
    print(f"{tokens} tokens in {a.steps} steps of {a.requests} requests (one more after a third of them): "
          f"{tokens / sum(map(len, got)):.2f} a request and step; {server.pages.free_pages} pages free")


if __name__ == "__main__":
    main()
