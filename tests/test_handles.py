"""A batch, a cache, a bank of adapters or a workspace whose fields are replaced: the next call gets the new
tensors' addresses and numbers, or refuses them, and so do copies.  No GPU needed: the library's entry points
are replaced by ones that note their arguments, and CPU tensors stand in for CUDA ones."""
import copy

import pytest

torch = pytest.importorskip("torch")

D, HKV, PAGE, PAGES = 64, 2, 16, 8
F16, I32 = torch.float16, torch.int32


class OnCard(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0

    def __deepcopy__(self, memo):
        return self.clone()


def card(*shape, dtype=F16):
    return real_zeros(*shape, dtype=dtype).as_subclass(OnCard)


real_zeros = torch.zeros


class Library:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in ("marlin_kv_append", "marlin_kv_read", "marlin_kv_attention", "marlin_lora_gemm"):
            return lambda *args: self.calls.append(args) or 0
        return getattr(self.real, name)


@pytest.fixture
def lib(monkeypatch):
    from w4a16_mixed_precision_gb300 import _binding, build
    build.build()
    library = Library(_binding.load())
    monkeypatch.setattr(_binding, "_lib", library)
    monkeypatch.setattr(_binding, "kv_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    monkeypatch.setattr(torch, "zeros", lambda *s, device=None, **k: real_zeros(*s, **k).as_subclass(OnCard))
    return library


def make():
    import w4a16_mixed_precision_gb300 as w4
    cache = w4.Kv4Cache(PAGES, HKV, D, PAGE, device="cuda:0")
    batch = w4.Kv4Batch(card(3, 4, dtype=I32), card(3, dtype=I32), card(4, dtype=I32), 5, 2)
    return w4, cache, batch, w4.Kv4Workspace(batch, 4, cache)


# places among marlin_kv_append's arguments
CACHE, N_PAGES, TABLE, MAX_PAGES, LENGTHS, START, REQUESTS, TOKENS, WORKSPACE = 6, 7, 11, 12, 13, 14, 15, 16, 17


def append(w4, lib, cache, batch, ws, tokens=5):
    k = card(tokens, HKV, D)
    w4.kv4_append(k, k, cache, batch, ws)
    return lib.calls[-1]


def test_replaced_tensors_of_a_batch(lib):
    w4, cache, batch, ws = make()
    append(w4, lib, cache, batch, ws)
    old = batch.page_table, batch.lengths, batch.q_start
    batch.page_table, batch.lengths, batch.q_start = card(2, 7, dtype=I32), card(2, dtype=I32), card(3, dtype=I32)
    a = append(w4, lib, cache, batch, ws)
    assert (a[TABLE], a[LENGTHS], a[START]) == tuple(t.data_ptr() for t in (batch.page_table, batch.lengths, batch.q_start))
    assert (a[MAX_PAGES], a[REQUESTS], a[TOKENS]) == (7, 2, 5)
    # attention and read get the same
    q = card(5, 4, D)
    w4.kv4_attention_into(q, cache, batch, ws, card(5, 4, D))
    assert batch.lengths.data_ptr() in lib.calls[-1] and old[1].data_ptr() not in lib.calls[-1]


def test_replaced_number_of_tokens(lib):
    w4, cache, batch, ws = make()
    batch.tokens, batch.max_q = 3, 1
    assert append(w4, lib, cache, batch, ws, tokens=3)[TOKENS] == 3
    w4.kv4_attention_into(card(3, 4, D), cache, batch, ws, card(3, 4, D))
    assert lib.calls[-1][4 + 5 + 6] == 1   # max_q
    with pytest.raises(ValueError):
        append(w4, lib, cache, batch, ws, tokens=5)
    batch.tokens = -1
    with pytest.raises(ValueError):
        append(w4, lib, cache, batch, ws, tokens=0)


@pytest.mark.parametrize("field,bad", [
    ("page_table", lambda: card(3, 4, dtype=torch.int64)), ("page_table", lambda: card(4, 3, dtype=I32).t()),
    ("page_table", lambda: card(2, 4, dtype=I32)), ("lengths", lambda: card(4, dtype=I32)),
    ("lengths", lambda: real_zeros(3, dtype=I32)), ("q_start", lambda: card(3, dtype=I32))])
def test_replacements_that_do_not_fit_are_refused(lib, field, bad):
    w4, cache, batch, ws = make()
    setattr(batch, field, bad())
    with pytest.raises(ValueError):
        append(w4, lib, cache, batch, ws)
    assert not lib.calls


def test_replaced_cache_and_workspace(lib):
    w4, cache, batch, ws = make()
    append(w4, lib, cache, batch, ws)
    cache.buf, ws.buf = card(cache.nbytes, dtype=torch.uint8), card(8192, dtype=torch.uint8)
    a = append(w4, lib, cache, batch, ws)
    assert (a[CACHE], a[WORKSPACE]) == (cache.buf.data_ptr(), ws.buf.data_ptr())
    w4.kv4_attention_into(card(5, 4, D), cache, batch, ws, card(5, 4, D))
    assert lib.calls[-1][-3:-1] == (ws.buf.data_ptr(), 8192)
    for change in (dict(buf=card(cache.nbytes - 1, dtype=torch.uint8)), dict(buf=real_zeros(cache.nbytes, dtype=torch.uint8)),
                   dict(buf=card(cache.nbytes), n_pages=PAGES), dict(buf=cache.buf, n_pages=PAGES + 1)):
        for name, value in change.items():
            setattr(cache, name, value)
        with pytest.raises(ValueError):
            append(w4, lib, cache, batch, ws)
    cache.n_pages = PAGES - 1   # fewer pages in the same buffer
    assert append(w4, lib, cache, batch, ws)[N_PAGES] == PAGES - 1


def test_replaced_adapters(lib):
    import w4a16_mixed_precision_gb300 as w4
    K, N, M = 256, 128, 2
    bank = w4.LoraBank(card(3, 8, K), card(3, N, 8), card(3, dtype=torch.float32))
    nbytes, off_s, off_z = w4.packed_layout(K, N, 128, False)
    w = w4.PackedWeights(card(nbytes, dtype=torch.uint8), K, N, 128, False, off_s, off_z)
    ws = w4.LoraWorkspace.__new__(w4.LoraWorkspace)
    ws.buf, ws.nbytes = card(64, dtype=torch.uint8), 64
    run = lambda: w4.lora_gemm_into(card(M, K), w, bank, card(M, dtype=I32), ws, card(M, N))  # noqa: E731
    run()
    a, b, scaling = 4, 5, 6
    assert lib.calls[-1][a:a + 3] == (bank.a.data_ptr(), bank.b.data_ptr(), bank.scaling.data_ptr())
    bank.a, bank.b, bank.scaling = card(5, 12, K), card(5, N, 12), card(5, dtype=torch.float32)
    run()
    assert lib.calls[-1][a:a + 3] == (bank.a.data_ptr(), bank.b.data_ptr(), bank.scaling.data_ptr())
    assert lib.calls[-1][8:10] == (5, 16) and bank.a.shape == (5, 16, K) and (bank.n, bank.r) == (5, 16)
    bank.a = card(5, 16, K + 64)
    with pytest.raises(ValueError):
        run()
    bank.a = card(5, 8, K)
    with pytest.raises(ValueError):
        run()
    with pytest.raises(AttributeError):
        bank.r = 8


def test_copies_have_their_own_addresses(lib):
    w4, cache, batch, ws = make()
    append(w4, lib, cache, batch, ws)
    bank = w4.LoraBank(card(3, 8, 256), card(3, 128, 8), card(3, dtype=torch.float32))
    c, b, s, k = copy.deepcopy((cache, batch, ws, bank))
    args = append(w4, lib, c, b, s)
    assert args[CACHE] == c.buf.data_ptr() != cache.buf.data_ptr()
    assert args[LENGTHS] == b.lengths.data_ptr() != batch.lengths.data_ptr()
    assert args[WORKSPACE] == s.buf.data_ptr() != ws.buf.data_ptr()
    assert (k._args or k._check())[0] == k.a.data_ptr() != bank.a.data_ptr()
