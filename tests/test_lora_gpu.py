"""Low-rank adapters beside the W4A16 product, against the oracle's product plus
the adapters' part in 64 bits.

Tolerance, derived: the base product's own (1e-2 + 2e-3 |y|, the parity tolerance
of the product) covers its rounding; the sum is rounded once more (2^-11 |y|);
v is rounded to fp16 relative to its row's largest component u (2^-11 u each),
which moves the adapters' part by at most 2^-11 u sum_j |B[n][j]|.
"""
import numpy as np
import pytest

import oracle
from workloads import Problem, make_inputs

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make(M, K, N, group, asym, r, n, seed, amp=1.0):
    import w4a16_mixed_precision_gb300 as w4
    inp = make_inputs(Problem("lora", M, K, N, group, asym))
    rng = np.random.default_rng(seed)
    a = (amp * rng.standard_normal((n, r, K)) / np.sqrt(K)).astype(np.float16)
    b = rng.standard_normal((n, N, r)).astype(np.float16)
    scaling = rng.uniform(0.5, 2.0, n).astype(np.float32)
    cu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    pw = w4.repack(cu(inp.Qp), cu(inp.S), cu(inp.Zp) if inp.Zp is not None else None, group)
    return inp, a, b, scaling, pw, w4.LoraBank(cu(a), cu(b), cu(scaling)), cu(inp.X)


def check(y, inp, a, b, scaling, index, group, N):
    base = oracle.w4a16(inp.X, inp.Qp, inp.S, inp.Zp, group, N)
    ref, extra = base.astype(np.float64).copy(), np.zeros(base.shape)
    for m, i in enumerate(index):
        if i >= 0:
            v = scaling[i].astype(np.float64) * (a[i].astype(np.float64) @ inp.X[m].astype(np.float64))
            ref[m] += b[i].astype(np.float64) @ v
            extra[m] = 2.0 ** -11 * np.abs(v).max() * np.abs(b[i].astype(np.float64)).sum(1)
    err = np.abs(y.astype(np.float64) - ref)
    tol = 1e-2 + 2e-3 * np.abs(base) + 2.0 ** -11 * np.abs(ref) + extra
    assert (err <= tol).all(), f"max error {err.max()}, {(err / tol).max():.2f} of the tolerance"
    # and the adapters' part itself is there: far closer to ref than the base product is
    rows = [m for m, i in enumerate(index) if i >= 0]
    if rows:
        assert np.linalg.norm(err[rows]) < 0.05 * np.linalg.norm((ref - base)[rows])


CASES = [
    # M, K, N, group, asym, r, adapters, index
    (1, 256, 128, 128, False, 8, 1, "zero"),
    (1, 4096, 384, 128, False, 16, 3, "zero"),
    (5, 1024, 256, 128, True, 16, 4, "random"),
    (16, 512, 640, 512, True, 24, 7, "random"),        # rank that is no power of two
    (17, 384, 256, 128, False, 32, 40, "own"),         # every row its own adapter
    (33, 1024, 384, 128, False, 64, 5, "runs"),
    (64, 512, 256, 128, True, 128, 3, "random"),
    (40, 512, 256, 128, False, 16, 2, "random"),       # several 16 rows of one adapter, in any places
    (127, 512, 384, 128, False, 64, 6, "random"),
    (127, 256, 128, 128, True, 48, 127, "own"),
    (90, 4096, 256, 128, False, 32, 30, "runs"),
    (130, 640, 256, 128, False, 16, 9, "random"),      # blocks of 32 rows, adapters in any order
    (300, 1024, 384, 128, False, 72, 4, "runs"),
    (257, 512, 256, 128, False, 8, 2, "none"),
    (128, 256, 128, 128, False, 40, 200, "own"),
    (256, 512, 128, 128, False, 16, 3, "random"),      # the most rows of one kernel, and one more
    (257, 512, 128, 128, False, 24, 3, "random"),
    (320, 256, 128, 128, False, 32, 400, "own"),       # more items than clusters
    (321, 512, 128, 128, False, 64, 9, "random"),
    (600, 512, 256, 128, False, 16, 30, "random"),
]


def index_of(kind, M, n, rng):
    if kind == "zero":
        return np.zeros(M, np.int32)
    if kind == "none":
        return np.full(M, -1, np.int32)
    if kind == "own":
        return (np.arange(M) % n).astype(np.int32)
    if kind == "runs":
        return (np.arange(M) // 13 % (n + 1) - 1).astype(np.int32)
    return rng.integers(-1, n, M).astype(np.int32)


@pytest.mark.parametrize("M,K,N,group,asym,r,n,kind", CASES)
def test_lora_gemm(M, K, N, group, asym, r, n, kind):
    import w4a16_mixed_precision_gb300 as w4
    inp, a, b, scaling, pw, bank, x = make(M, K, N, group, asym, r, n, seed=M + r)
    index = index_of(kind, M, n, np.random.default_rng(M))
    ws = w4.LoraWorkspace(M, K, N, group, r)
    di = torch.from_numpy(index).cuda()
    y = w4.lora_gemm(x, pw, bank, di, ws)
    again = w4.lora_gemm(x, pw, bank, di, ws)
    assert w4.device_status(ws) == 0
    assert torch.equal(y, again)
    check(y.cpu().numpy(), inp, a, b, scaling, index, group, N)
    # rows without an adapter are the product's, bit for bit
    base = w4.gemm(x, pw, w4.Workspace(M, K, N, group))
    none = torch.from_numpy(index < 0).cuda()
    assert torch.equal(y[none], base[none])


def test_workspace_serves_fewer_rows_and_padded_ranks():
    import w4a16_mixed_precision_gb300 as w4
    K, N, g, r, n = 512, 256, 128, 12, 3   # rank 12 is padded to 16
    ws = w4.LoraWorkspace(200, K, N, g, r)
    for M in (200, 1, 130, 31, 127, 128):
        inp, a, b, scaling, pw, bank, x = make(M, K, N, g, False, r, n, seed=M)
        assert bank.r == 16
        index = index_of("random", M, n, np.random.default_rng(M))
        y = w4.lora_gemm(x, pw, bank, torch.from_numpy(index).cuda(), ws)
        assert w4.device_status(ws) == 0
        check(y.cpu().numpy(), inp, a, b, scaling, index, g, N)


def test_stack_of_different_ranks():
    import w4a16_mixed_precision_gb300 as w4
    M, K, N, g = 9, 512, 256, 128
    inp, a, b, scaling, pw, _, x = make(M, K, N, g, False, 16, 2, seed=4)
    cu = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
    bank = w4.LoraBank.stack([(cu(a[0]), cu(b[0]), scaling[0]), (cu(a[1, :5]), cu(b[1, :, :5]), scaling[1])])
    a[1, 5:] = 0
    index = (np.arange(M) % 3 - 1).astype(np.int32)
    y = w4.lora_gemm(x, pw, bank, cu(index), w4.LoraWorkspace(M, K, N, g, bank.r))
    check(y.cpu().numpy(), inp, a, b, scaling, index, g, N)


@pytest.mark.parametrize("amp", [1e-4, 3e4])
def test_magnitudes_of_v_beyond_fp16(amp):
    """x . A^T above fp16's largest number and far below its normal range: the rows' powers of two carry it."""
    import w4a16_mixed_precision_gb300 as w4
    M, K, N, g, r, n = 7, 512, 128, 128, 16, 2
    inp, a, b, scaling, pw, _, x = make(M, K, N, g, False, r, n, seed=5, amp=min(amp, 2e3))
    scaling *= np.float32(amp)
    b = (b / np.float32(np.clip(amp, 1e-3, 4e3))).astype(np.float16)
    cu = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
    bank = w4.LoraBank(cu(a), cu(b), cu(scaling))
    index = np.zeros(M, np.int32)
    y = w4.lora_gemm(x, pw, bank, cu(index), w4.LoraWorkspace(M, K, N, g, r)).cpu().numpy().astype(np.float64)
    base = oracle.w4a16(inp.X, inp.Qp, inp.S, inp.Zp, g, N).astype(np.float64)
    v = scaling[0].astype(np.float64) * (inp.X.astype(np.float64) @ a[0].astype(np.float64).T)
    ref = base + v @ b[0].astype(np.float64).T
    tol = (1e-2 + 2e-3 * np.abs(base) + 2.0 ** -11 * np.abs(ref)
           + 2.0 ** -11 * np.abs(v).max(1, keepdims=True) * np.abs(b[0].astype(np.float64)).sum(1))
    fits = np.abs(ref) < 65000
    assert fits.any() and (np.abs(y - ref) <= tol)[fits].all()


def test_bad_adapter_is_reported_and_gives_none():
    import w4a16_mixed_precision_gb300 as w4
    M, K, N, g, r, n = 20, 256, 128, 128, 8, 2
    inp, a, b, scaling, pw, bank, x = make(M, K, N, g, False, r, n, seed=6)
    index = np.zeros(M, np.int32)
    index[3], index[17] = n, -1000
    ws = w4.LoraWorkspace(M, K, N, g, r)
    y = w4.lora_gemm(x, pw, bank, torch.from_numpy(index).cuda(), ws)
    assert w4.device_status(ws) == 7
    index[3] = -1
    check(y.cpu().numpy(), inp, a, b, scaling, index, g, N)


def test_nan_stays_in_its_row():
    import w4a16_mixed_precision_gb300 as w4
    M, K, N, g, r, n = 18, 256, 128, 128, 8, 2
    inp, a, b, scaling, pw, bank, x = make(M, K, N, g, False, r, n, seed=7)
    x[4, 9] = float("nan")
    index = torch.zeros(M, dtype=torch.int32, device="cuda")
    y = w4.lora_gemm(x, pw, bank, index, w4.LoraWorkspace(M, K, N, g, r))
    bad = torch.isnan(y)
    assert bool(bad[4].all()) and int(bad.sum()) == N


def test_refusals():
    import w4a16_mixed_precision_gb300 as w4
    M, K, N, g, r, n = 4, 256, 128, 128, 8, 2
    _, a, b, scaling, pw, bank, x = make(M, K, N, g, False, r, n, seed=8)
    cu = lambda t: torch.from_numpy(np.ascontiguousarray(t)).cuda()  # noqa: E731
    ws = w4.LoraWorkspace(M, K, N, g, r)
    index = torch.zeros(M, dtype=torch.int32, device="cuda")
    for bad in ((x.float(), index), (x, index.long()), (x[:, :128].contiguous(), index), (x, index[:3]),
                (x, index.cpu())):
        with pytest.raises(ValueError):
            w4.lora_gemm(bad[0], pw, bank, bad[1], ws)
    for args in ((cu(a), cu(b[:1]), cu(scaling)), (cu(a).float(), cu(b), cu(scaling)), (cu(a), cu(b), cu(scaling)[:1]),
                 (cu(a), cu(b[:, :, :4]), cu(scaling)), (torch.from_numpy(a), cu(b), cu(scaling))):
        with pytest.raises(ValueError):
            w4.LoraBank(*args)
    with pytest.raises(ValueError):
        w4.LoraBank(torch.zeros((1, 136, K), dtype=torch.float16, device="cuda"),
                    torch.zeros((1, N, 136), dtype=torch.float16, device="cuda"), cu(scaling)[:1])
    with pytest.raises(ValueError):
        w4.LoraBank.stack([])
    small = w4.LoraWorkspace(1, K, N, g, r)
    big = torch.zeros((600, K), dtype=torch.float16, device="cuda")
    with pytest.raises(w4.MarlinError) as e:
        w4.lora_gemm(big, pw, bank, torch.zeros(600, dtype=torch.int32, device="cuda"), small)
    assert e.value.status == 4
    assert w4.lora_gemm(x[:0], pw, bank, index[:0], ws).shape == (0, N)
