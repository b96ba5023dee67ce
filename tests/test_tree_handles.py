"""A rope, a batch, caches or a workspace whose fields are replaced, for the entry points of drafted trees: the next
call gets the new tensors' addresses and numbers, or refuses them.  No GPU needed: as in test_handles.py."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_handles import D, F16, HKV, I32, PAGE, PAGES, card, make, real_zeros  # noqa: E402, F401
from test_handles import Library as Base  # noqa: E402

NAMES = ("marlin_kv_rope_append", "marlin_kv_tree", "marlin_kv_tree_attention")


class Library(Base):
    def __getattr__(self, name):
        if name in ("marlin_kv_compact", "marlin_kv_copy_pages"):  # the caches' addresses: the array lives as long as the call
            return lambda at, n, *args: self.calls.append((*(ctypes.c_uint64 * n).from_address(at), n, *args)) or 0
        if name in NAMES:
            return lambda *args: self.calls.append(args) or 0
        return super().__getattr__(name)


@pytest.fixture
def lib(monkeypatch):
    from test_handles import OnCard
    from w4a16_mixed_precision_gb300 import _binding, build
    build.build()
    library = Library(_binding.load())
    monkeypatch.setattr(_binding, "_lib", library)
    monkeypatch.setattr(_binding, "kv_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    monkeypatch.setattr(torch, "zeros", lambda *s, device=None, **k: real_zeros(*s, **k).as_subclass(OnCard))
    monkeypatch.setattr(torch, "empty", lambda *s, device=None, **k: real_zeros(*s, **k).as_subclass(OnCard))
    return library


def rope_of(w4, rows, rot, **k):
    return w4.Kv4Rope(card(rows, rot // 2, dtype=torch.float32), card(rows, rot // 2, dtype=torch.float32), **k)


def test_rope(lib):
    w4, cache, batch, ws = make()
    rope = rope_of(w4, 9, D)
    q, k, out, pos = card(5, 4, D), card(5, HKV, D), card(5, 4, D), card(5, dtype=I32)
    run = lambda pos=pos: w4.kv4_rope_append_into(q, k, k, pos, rope, cache, batch, ws, out) is out and lib.calls[-1]  # noqa: E731
    a = run()
    TABLE, ROWS, ROT, AXES = 12, 13, 14, 11
    assert (a[TABLE], a[ROWS], a[ROT], a[AXES]) == (rope.table.data_ptr(), 9, D, 1)
    assert a[16] == bytes(D // 2) and a[17] == out.data_ptr() and a[20] == cache.buf.data_ptr()
    rope.table = card(20, D // 2, 2, dtype=torch.float32)
    a = run()
    assert (a[TABLE], a[ROWS]) == (rope.table.data_ptr(), 20)
    rope.axes = (0, 2) * (D // 4)
    with pytest.raises(ValueError):
        run()                                    # positions of one axis
    assert run(card(3, 5, dtype=I32))[AXES] == 3 and lib.calls[-1][16] == bytes((0, 2)) * (D // 4)
    for field, bad in (("axes", (0,) * 3), ("axes", (4,) * (D // 2)), ("rot", D // 2), ("table", card(20, D // 2, 2)),
                       ("table", real_zeros(20, D // 2, 2)), ("table", card(0, D // 2, 2, dtype=torch.float32))):
        old = getattr(rope, field)
        setattr(rope, field, bad)
        with pytest.raises(ValueError):
            run(card(3, 5, dtype=I32))
        setattr(rope, field, old)
    batch.tokens = 4
    with pytest.raises(ValueError):
        run(card(3, 5, dtype=I32))


def test_tree_and_its_attention(lib):
    w4, cache, batch, ws = make()
    parents = card(5, dtype=I32)
    mask, positions = w4.kv4_tree(parents, batch, ws)
    assert lib.calls[-1][:6] == (parents.data_ptr(), batch.lengths.data_ptr(), batch.q_start.data_ptr(), 3, 5, 1)
    assert mask.shape == (5, 1) and positions.shape == (5,)
    batch.max_q = 33
    assert w4.kv4_tree(parents, batch, ws)[0].shape == (5, 2) and lib.calls[-1][5] == 2
    batch.lengths = card(3, dtype=I32)
    q, tree = card(5, 4, D), card(5, 7, dtype=I32)
    w4.kv4_tree_attention_into(q, cache, batch, tree, ws, card(5, 4, D), window=3)
    a = lib.calls[-1]
    assert batch.lengths.data_ptr() in a and a[15:18] == (33, tree.data_ptr(), 7) and a[19] == 3
    for bad in (card(4, 7, dtype=I32), card(5, 7, dtype=torch.int64), card(5, dtype=I32), real_zeros(5, 7, dtype=I32),
                card(7, 5, dtype=I32).t()):
        with pytest.raises(ValueError):
            w4.kv4_tree_attention_into(q, cache, batch, bad, ws, card(5, 4, D))


def test_caches_of_several_layers(lib):
    w4, cache, batch, ws = make()
    more = [w4.Kv4Cache(PAGES, HKV, D, PAGE, device="cuda:0") for _ in range(3)]
    index, kept = card(5, dtype=I32), card(3, dtype=I32)
    w4.kv4_compact(more, batch, index, kept, ws)
    assert lib.calls[-1][:8] == (*(c.buf.data_ptr() for c in more), 3, PAGES, HKV, D, PAGE)
    more[1].buf = card(more[1].nbytes, dtype=torch.uint8)
    pairs = card(2, dtype=I32)
    w4.kv4_copy_pages(tuple(more), pairs, pairs, ws)
    assert lib.calls[-1][:4] == (*(c.buf.data_ptr() for c in more), 3)
    w4.kv4_copy_pages(cache, pairs, pairs, ws)
    assert lib.calls[-1][:2] == (cache.buf.data_ptr(), 1)
    more[2].n_pages = PAGES - 1
    for go in (lambda c: w4.kv4_compact(c, batch, index, kept, ws), lambda c: w4.kv4_copy_pages(c, pairs, pairs, ws)):
        for bad in (more, [], ()):
            with pytest.raises(ValueError):
                go(bad)
