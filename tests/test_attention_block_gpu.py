"""The operators together, as examples/attention_block.py runs them: against the same block in plain
torch operations in 64 bits on the values that the kernels read (the 4-bit weights' fp16 values, the
cache's values as kv4_read returns them).

Tolerance: 2 % of an output row's norm.  The QKV product and the attention output are rounded to fp16
(2^-11 each) and the output product passes them on, in 2^-11 steps again; 2 % leaves room for a few
such roundings and is a tenth of what a wrong adapter, head or position would change.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    sys.path.insert(0, os.path.join(ROOT, "examples"))


def weights(pw, ws):
    """The fp16 values of the weights, by multiplying the identity."""
    import w4a16_mixed_precision_gb300 as w4
    eye = torch.eye(pw.K, dtype=torch.float16, device="cuda")
    return torch.cat([w4.gemm(e.contiguous(), pw, ws) for e in eye.split(128)]).double()


def project(x, W, bank, adapter):
    y = x.double() @ W
    for m, a in enumerate(adapter.tolist()):
        if a >= 0:
            y[m] += bank.scaling[a].double() * ((x[m].double() @ bank.a[a].double().t()) @ bank.b[a].double().t())
    return y


def test_block_matches_plain():
    import attention_block as ab
    import w4a16_mixed_precision_gb300 as w4
    hidden, heads, hkv, prompts, steps, seed = 512, 8, 2, (150, 7, 64), 3, 3
    outs, block, requests = ab.serve(hidden, heads, hkv, prompts, steps, rank=8, page_size=16, seed=seed)
    d, G = hidden // heads, heads // hkv
    big = w4.Workspace(128, hidden, block.qkv.N, 128)
    Wq, Wo = weights(block.qkv, big), weights(block.out, w4.Workspace(128, hidden, hidden, 128))
    # every cached value at the end; earlier calls saw a prefix of it
    count = len(prompts)
    start = [0]
    for n in requests.lengths:
        start.append(start[-1] + n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = w4.kv4_read(block.cache, w4.Kv4Batch(requests.table, i32(requests.lengths), i32(start), start[-1], max(requests.lengths)),
                         block.kv_ws)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    for call in range(steps + 1):
        new = prompts if call == 0 else [1] * count
        x = torch.randn((sum(new), hidden), generator=gen, device="cuda").half()
        adapter = torch.arange(-1, count - 1, device="cuda").repeat_interleave(torch.tensor(new, device="cuda"))
        q = project(x, Wq, block.qkv_adapters, adapter)[:, :hidden].view(-1, heads, d)
        rows, at = [], 0
        for b in range(count):
            k, v = kc[start[b]:start[b + 1]].double(), vc[start[b]:start[b + 1]].double()
            first = 0 if call == 0 else prompts[b] + call - 1
            for i in range(new[b]):
                n = first + i + 1
                s = torch.einsum("hd,nhd->hn", q[at], k[:n].repeat_interleave(G, 1)) / d ** 0.5
                rows.append(torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v[:n].repeat_interleave(G, 1)).flatten())
                at += 1
        ref = project(torch.stack(rows), Wo, block.out_adapters, adapter)
        err = (outs[call].double() - ref).norm(dim=1) / ref.norm(dim=1)
        assert float(err.max()) < 0.02, (call, float(err.max()))
