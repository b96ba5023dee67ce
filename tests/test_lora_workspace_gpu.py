"""One workspace for adapters' calls of many row counts and for the plain product: every call leaves
it zero (the product's reducers take a non-zero word for a sum that has been written), and gives the
bits that it gives with a workspace of its own."""
import pytest

from test_lora_gpu import _built  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def inputs(K, N, r, n, seed):
    import w4a16_mixed_precision_gb300 as w4
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-2**31, 2**31, (K // 8, N), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s = (0.02 * (0.5 + torch.rand((K // 128, N), generator=g, device="cuda"))).half()
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    bank = w4.LoraBank((normal(n, r, K) / K ** 0.5).half(), normal(n, N, r).half(), torch.ones(n, device="cuda"))
    return w4.repack(q, s, None, 128), bank, lambda M: (normal(M, K).half(), torch.randint(
        -1, n, (M,), generator=g, device="cuda", dtype=torch.int32))


@pytest.mark.parametrize("K,N,r,rows", [
    (11008, 4096, 16, (300, 768, 257, 768, 40, 600)),
    (4096, 12288, 16, (400, 1024, 330, 2048, 1, 400)),
    (512, 384, 128, (321, 1280, 500, 129)),              # 384 columns: warps without any
    (256, 128, 40, (1000, 333, 512)),
])
def test_one_workspace_for_many_row_counts(K, N, r, rows):
    import w4a16_mixed_precision_gb300 as w4
    pw, bank, make = inputs(K, N, r, 5, seed=K + r)
    ws = w4.LoraWorkspace(max(rows), K, N, 128, r)
    for M in rows:
        x, index = make(M)
        y = w4.lora_gemm(x, pw, bank, index, ws)
        assert int(ws.buf.count_nonzero()) == 0, M
        own = w4.LoraWorkspace(M, K, N, 128, r)
        assert torch.equal(y, w4.lora_gemm(x, pw, bank, index, own)), M
        base = w4.gemm(x, pw, ws)
        assert int(ws.buf.count_nonzero()) == 0, M
        assert torch.equal(base, w4.gemm(x, pw, w4.Workspace(M, K, N, 128))), M
        none = index < 0
        assert torch.equal(y[none], base[none]), M
        # once more, with the queue full: what a call zeroes, the next one finds zero
        assert all(torch.equal(w4.lora_gemm(x, pw, bank, index, ws), y) for _ in range(3)), M
    assert w4.device_status(ws) == 0


def test_one_workspace_for_two_shapes():
    """The largest of two shapes' workspaces serves both, in turn."""
    import w4a16_mixed_precision_gb300 as w4
    shapes = [(1024, 4096, 16, 400), (4096, 1024, 64, 700)]
    ws = max((w4.LoraWorkspace(M, K, N, 128, r) for K, N, r, M in shapes), key=lambda w: w.nbytes)
    for turn in range(2):
        for K, N, r, M in shapes:
            pw, bank, make = inputs(K, N, r, 3, seed=N + turn)
            x, index = make(M)
            y = w4.lora_gemm(x, pw, bank, index, ws)
            assert int(ws.buf.count_nonzero()) == 0
            assert torch.equal(y, w4.lora_gemm(x, pw, bank, index, w4.LoraWorkspace(M, K, N, 128, r)))
    assert w4.device_status(ws) == 0
