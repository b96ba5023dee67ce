"""Host-side argument checks of the adapter and cache entry points (no GPU needed:
these paths return before any CUDA call)."""
import ctypes

import pytest

G = 0x10000  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    from w4a16_mixed_precision_gb300 import _binding, build
    build.build()
    return _binding.load()


def lora(lib, X=G, packed=G, scales=G, zeros=None, A=G, B=G, scaling=G, index=G, adapters=2, r=16, Y=G, M=4, K=256,
         N=256, group=128, ws=G, ws_bytes=0):
    return lib.marlin_lora_gemm(X, packed, scales, zeros, A, B, scaling, index, adapters, r, Y, M, K, N, group, ws,
                                ws_bytes, None)


def test_lora_checks(lib):
    from w4a16_mixed_precision_gb300 import _binding as b
    assert lora(lib, M=0) == b.OK
    for bad in (dict(M=-1), dict(r=0), dict(adapters=0), dict(K=200), dict(N=64), dict(group=96), dict(X=None),
                dict(A=None), dict(B=None), dict(scaling=None), dict(index=None), dict(Y=None), dict(ws=None)):
        assert lora(lib, **bad) == b.ERR_INVALID_ARG, bad
    for bad in (dict(r=12), dict(r=136), dict(group=64)):
        assert lora(lib, **bad) == b.ERR_UNSUPPORTED, bad
    for bad in (dict(A=G + 8), dict(B=G + 2), dict(Y=G + 8), dict(scaling=G + 2), dict(index=G + 1), dict(zeros=G + 4)):
        assert lora(lib, **bad) == b.ERR_MISALIGNED, bad


def copy(lib, name, k=G, v=G, cache=G, n_pages=4, hkv=2, D=128, page=16, table=G, max_pages=8, lens=G, q_start=G,
         B=3, T=5, ws=G, strides=(256, 128)):
    kv = (cache, n_pages, hkv, D, page, table, max_pages, lens, q_start, B, T, ws, None)
    if name == "append":
        return lib.marlin_kv_append(k, *strides, v, *strides, *kv)
    return lib.marlin_kv_read(k, v, *kv)


@pytest.mark.parametrize("name", ["append", "read"])
def test_append_and_read_checks(lib, name):
    from w4a16_mixed_precision_gb300 import _binding as b
    assert copy(lib, name, B=0) == b.OK and copy(lib, name, T=0) == b.OK
    for bad in (dict(k=None), dict(v=None), dict(cache=None), dict(table=None), dict(lens=None), dict(q_start=None),
                dict(ws=None), dict(B=-1), dict(T=-1), dict(max_pages=0), dict(n_pages=0), dict(hkv=0), dict(D=0), dict(page=0)):
        assert copy(lib, name, **bad) == b.ERR_INVALID_ARG, bad
    for bad in (dict(D=96), dict(D=256), dict(page=24), dict(page=1040), dict(page=1024, max_pages=(1 << 20) + 1)):
        assert copy(lib, name, **bad) == b.ERR_UNSUPPORTED, bad
    for bad in (dict(cache=G + 8), dict(table=G + 2), dict(lens=G + 1), dict(q_start=G + 2), dict(ws=G + 4), dict(k=G + 8)):
        assert copy(lib, name, **bad) == b.ERR_MISALIGNED, bad
    if name == "append":
        for strides in ((252, 128), (256, 124), (-256, 128)):
            assert copy(lib, name, strides=strides) == b.ERR_MISALIGNED


def attention(lib, q=G, heads=4, hkv=2, D=128, page=16, B=3, T=5, max_q=2, scale=0.1, window=0, out=G, ws=G, strides=(512, 128)):
    return lib.marlin_kv_attention(q, *strides, heads, G, 4, hkv, D, page, G, 8, G, G, B, T, max_q, scale, window, out, ws,
                                   0, None)


def test_attention_checks(lib):
    from w4a16_mixed_precision_gb300 import _binding as b
    assert attention(lib, B=0) == b.OK and attention(lib, T=0) == b.OK
    for bad in (dict(heads=3), dict(heads=0), dict(hkv=0), dict(window=-1), dict(max_q=-1), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(q=None), dict(out=None), dict(ws=None)):
        assert attention(lib, **bad) == b.ERR_INVALID_ARG, bad
    for bad in (dict(D=80), dict(page=40)):
        assert attention(lib, **bad) == b.ERR_UNSUPPORTED, bad
    for bad in (dict(q=G + 8), dict(out=G + 8), dict(ws=G + 8), dict(strides=(516, 128)), dict(strides=(512, 132))):
        assert attention(lib, **bad) == b.ERR_MISALIGNED, bad


def test_sizes(lib):
    from w4a16_mixed_precision_gb300 import _binding as b
    assert b.kv_cache_bytes(3, 8, 128, 64) == 3 * 8 * 64 * (128 + 8)
    assert b.kv_cache_bytes(1, 1, 64, 16) == 16 * 72
    assert b.kv_cache_bytes(100000, 8, 128, 64) == 100000 * 8 * 64 * 136   # past 32 bits
    for args, status in (((3, 8, 128, 20), b.ERR_UNSUPPORTED), ((3, 8, 32, 16), b.ERR_UNSUPPORTED), ((0, 8, 128, 16), b.ERR_INVALID_ARG)):
        with pytest.raises(b.MarlinError) as e:
            b.kv_cache_bytes(*args)
        assert e.value.status == status
    n = ctypes.c_size_t()
    assert lib.marlin_kv_workspace_bytes(4, 3, 128, 1, 1, 0, ctypes.byref(n)) == b.ERR_INVALID_ARG
    assert lib.marlin_kv_workspace_bytes(4, 2, 96, 1, 1, 0, ctypes.byref(n)) == b.ERR_UNSUPPORTED
    assert lib.marlin_kv_workspace_bytes(4, 2, 128, -1, 1, 0, ctypes.byref(n)) == b.ERR_INVALID_ARG
    assert lib.marlin_kv_cache_bytes(1, 1, 64, 16, None) == b.ERR_INVALID_ARG
    assert lib.marlin_lora_workspace_bytes(4, 256, 256, 128, 12, 0, ctypes.byref(n)) == b.ERR_UNSUPPORTED
    assert lib.marlin_lora_workspace_bytes(4, 256, 256, 128, 0, 0, ctypes.byref(n)) == b.ERR_INVALID_ARG


def test_batch_checks():
    """Kv4Batch and LoraBank refuse what does not fit before they reach the library."""
    torch = pytest.importorskip("torch")
    import w4a16_mixed_precision_gb300 as w4
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.Kv4Batch(t, torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 2, 1)   # not on a GPU
    h = torch.zeros((1, 8, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        w4.LoraBank(h, torch.zeros((1, 32, 8), dtype=torch.float16), torch.ones(1))
    with pytest.raises(ValueError):
        w4.LoraBank(h, torch.zeros((2, 32, 8), dtype=torch.float16), torch.ones(2))
