"""One attention block of a served model, as a decode loop would run it: 4-bit QKV and output
projections with each request's low-rank adapter beside them, keys and values in a 4-bit paged
cache, attention over it.  Random weights; rotary embedding is left out.

    python examples/attention_block.py            # 6 requests: their prompts, then 16 steps

`AttentionBlock.forward` takes a batch of any mix of prompts and single tokens; `Requests` deals out
the cache's pages and keeps the lengths.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import w4a16_mixed_precision_gb300 as w4


def random_projection(K: int, N: int, gen: torch.Generator, group: int = 128):
    q = torch.randint(-2**31, 2**31, (K // 8, N), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    s = ((0.5 + torch.rand((K // group, N), generator=gen, device="cuda")) * (0.25 / K ** 0.5)).half()
    return w4.repack(q, s, None, group)


def random_adapters(n: int, r: int, K: int, N: int, gen: torch.Generator):
    a = torch.randn((n, r, K), generator=gen, device="cuda") / K ** 0.5
    b = torch.randn((n, N, r), generator=gen, device="cuda") * 0.1
    return w4.LoraBank(a.half(), b.half(), torch.ones(n, device="cuda"))


class Requests:
    """The cache's pages and lengths of a fixed number of requests."""

    def __init__(self, count: int, max_len: int, page_size: int):
        self.page_size, self.count = page_size, count
        self.pages = -(-max_len // page_size)
        # every request may grow to max_len; a server would deal pages out as they are needed
        order = torch.randperm(count * self.pages).to(torch.int32)
        self.table = order.view(count, self.pages).cuda()
        self.lengths = [0] * count

    def batch(self, new_tokens) -> w4.Kv4Batch:
        """new_tokens[b] more tokens for request b (0 for none)."""
        start = [0]
        for b, n in enumerate(new_tokens):
            self.lengths[b] += n
            start.append(start[-1] + n)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return w4.Kv4Batch(self.table, i32(self.lengths), i32(start), start[-1], max(new_tokens))


class AttentionBlock:
    def __init__(self, hidden: int, heads: int, kv_heads: int, requests: Requests, adapters: int, rank: int,
                 max_tokens: int, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.d = heads, kv_heads, hidden // heads
        n_qkv = (heads + 2 * kv_heads) * self.d
        self.qkv, self.out = random_projection(hidden, n_qkv, gen), random_projection(heads * self.d, hidden, gen)
        self.qkv_adapters = random_adapters(adapters, rank, hidden, n_qkv, gen)
        self.out_adapters = random_adapters(adapters, rank, heads * self.d, hidden, gen)
        self.qkv_ws = w4.LoraWorkspace(max_tokens, hidden, n_qkv, 128, rank)
        self.out_ws = w4.LoraWorkspace(max_tokens, heads * self.d, hidden, 128, rank)
        self.cache = w4.Kv4Cache(requests.count * requests.pages, kv_heads, self.d, requests.page_size)
        self.kv_ws = None

    def forward(self, x: torch.Tensor, batch: w4.Kv4Batch, adapter: torch.Tensor) -> torch.Tensor:
        """x fp16 [tokens, hidden], adapter int32 [tokens] (negative for none)."""
        if self.kv_ws is None:  # the first batch is the largest: the prompts
            self.kv_ws = w4.Kv4Workspace(batch, self.heads, self.cache)
        y = w4.lora_gemm(x, self.qkv, self.qkv_adapters, adapter, self.qkv_ws)
        q, k, v = (t.unflatten(1, (-1, self.d)) for t in
                   y.split([self.heads * self.d, self.kv_heads * self.d, self.kv_heads * self.d], dim=1))
        w4.kv4_append(k, v, self.cache, batch, self.kv_ws)
        o = w4.kv4_attention(q, self.cache, batch, self.kv_ws)
        return w4.lora_gemm(o.flatten(1), self.out, self.out_adapters, adapter, self.out_ws)


def serve(hidden=4096, heads=32, kv_heads=8, prompts=(700, 33, 1200, 64, 5, 512), steps=16, rank=16, page_size=64, seed=0):
    """The requests' prompts in one batch, then `steps` single tokens each; returns the outputs of every
    call, the block and the requests."""
    count, T = len(prompts), sum(prompts)
    requests = Requests(count, max(prompts) + steps, page_size)
    block = AttentionBlock(hidden, heads, kv_heads, requests, adapters=count - 1, rank=rank, max_tokens=T, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    of_request = torch.arange(-1, count - 1, dtype=torch.int32, device="cuda")  # request 0 has no adapter
    adapter = of_request.repeat_interleave(torch.tensor(prompts, device="cuda"))
    outs = [block.forward(torch.randn((T, hidden), generator=gen, device="cuda").half(), requests.batch(prompts), adapter)]
    for _ in range(steps):
        x = torch.randn((count, hidden), generator=gen, device="cuda").half()
        outs.append(block.forward(x, requests.batch([1] * count), of_request))
    for name, ws in (("qkv", block.qkv_ws), ("cache", block.kv_ws), ("out", block.out_ws)):
        status = w4.device_status(ws)
        if status:
            raise RuntimeError(f"{name}: {w4.status_string(status)}")
    return outs, block, requests


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    a = ap.parse_args()
    serve(a.hidden, a.heads, a.kv_heads, steps=2)  # builds nothing, but loads the kernels
    torch.cuda.synchronize()
    t = time.perf_counter()
    outs, block, requests = serve(a.hidden, a.heads, a.kv_heads, steps=a.steps)
    torch.cuda.synchronize()
    print(f"{len(outs)} calls ({outs[0].shape[0]} prompt tokens, then {a.steps} steps of {len(requests.lengths)} requests), "
          f"set-up included, in {time.perf_counter() - t:.3f} s; cache {block.cache.nbytes / 2**20:.1f} MiB "
          f"({16 * block.d / (4 * block.d + 32):.2f}x smaller than fp16)")


if __name__ == "__main__":
    main()
