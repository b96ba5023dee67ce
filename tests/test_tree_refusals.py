"""Calls for drafted trees that are refused before anything is launched: outputs whose rows overlap, odd numbers of
rotated channels; and caches in any iterable.  No GPU needed: as in test_handles.py and test_tree_ops_abi.py."""
import pytest

torch = pytest.importorskip("torch")

from test_handles import D, HKV, I32, PAGE, PAGES, card, make  # noqa: E402
from test_tree_handles import lib, rope_of  # noqa: E402, F401
from test_tree_ops_abi import check, rope  # noqa: E402
from test_tree_ops_abi import lib as real_lib  # noqa: E402, F401


def test_rotated_queries_that_overlap_are_refused(real_lib):  # noqa: F811
    """Two rows of q_out in the same place would hold whichever came last.  (Of the calls that are taken T is 0 or B is:
    nothing is launched.)"""
    check(rope, real_lib,
          invalid=[dict(out_strides=(0, 128)), dict(out_strides=(512, 0)), dict(out_strides=(0, 0)), dict(out_strides=(504, 128)),
                   dict(out_strides=(512, 120)), dict(out_strides=(128, 512)), dict(out_strides=(1024, 64)),
                   dict(heads=1, hkv=1, out_strides=(0, 128)), dict(T=1, out_strides=(0, 0))],
          ok=[dict(B=0, out_strides=(0, 0)), dict(T=0, out_strides=(0, 0))])


def test_layouts_that_do_not_overlap_are_taken(real_lib):  # noqa: F811
    """Tokens or heads outermost, one head, one token: these pass the check on overlaps, so that the next one (a misaligned
    table) answers."""
    check(rope, real_lib,
          misaligned=[dict(table=257 * 8, out_strides=s, **more) for s, more in (
              ((512, 128), {}), ((768, 128), {}), ((128, 640), {}), ((1024, 256), {}), ((136, 680), {}),
              ((128, 0), dict(heads=1, hkv=1)), ((0, 128), dict(T=1)), ((0, 0), dict(T=1, heads=1, hkv=1)))])


def test_out_with_overlapping_rows(lib):  # noqa: F811
    w4, cache, batch, ws = make()
    r = rope_of(w4, 9, D)
    q, k, pos = card(5, 4, D), card(5, HKV, D), card(5, dtype=I32)
    run = lambda out: w4.kv4_rope_append_into(q, k, k, pos, r, cache, batch, ws, out)  # noqa: E731
    for bad in (card(1, 4, D).expand(5, 4, D), card(5, 1, D).expand(5, 4, D), card(D).expand(5, 4, D),
                card(5 * 4 * D).as_strided((5, 4, D), (3 * D, D, 1))):
        with pytest.raises(ValueError):
            run(bad)
    n = len(lib.calls)
    for good in (card(5, 4, D), card(4, 5, D).transpose(0, 1), card(5, 6, D)[:, 1:5], card(5, 4, 2 * D)[..., :D], q):
        assert run(good) is good
    assert len(lib.calls) == n + 5


def test_odd_numbers_of_rotated_channels():
    import w4a16_mixed_precision_gb300 as w4
    for rot in (63, 1, 0, -2):
        with pytest.raises(ValueError):
            w4.Kv4Rope.from_theta(rot, 10, device="cuda:0")


def test_caches_in_any_iterable(lib):  # noqa: F811
    w4, cache, batch, ws = make()
    more = [w4.Kv4Cache(PAGES, HKV, D, PAGE, device="cuda:0") for _ in range(3)]
    index, kept, pairs = card(5, dtype=I32), card(3, dtype=I32), card(2, dtype=I32)
    at = tuple(c.buf.data_ptr() for c in more)
    for caches in (more, tuple(more), (c for c in more), dict(enumerate(more)).values()):
        w4.kv4_compact(caches, batch, index, kept, ws)
        assert lib.calls[-1][:4] == (*at, 3)
    w4.kv4_copy_pages(iter(more), pairs, pairs, ws)
    assert lib.calls[-1][:4] == (*at, 3)
    for go in (lambda c: w4.kv4_compact(c, batch, index, kept, ws), lambda c: w4.kv4_copy_pages(c, pairs, pairs, ws)):
        with pytest.raises(ValueError):
            go(iter(()))
