"""Host-side argument checks of the entry points for drafted trees, and who holds which page (no GPU needed: these paths
return before any CUDA call)."""
import ctypes
import random

import pytest

G = 0x10000  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    from w4a16_mixed_precision_gb300 import _binding, build
    build.build()
    return _binding.load()


def check(call, lib, invalid=(), unsupported=(), misaligned=(), ok=()):
    from w4a16_mixed_precision_gb300 import _binding as b
    for cases, status in ((invalid, b.ERR_INVALID_ARG), (unsupported, b.ERR_UNSUPPORTED), (misaligned, b.ERR_MISALIGNED), (ok, b.OK)):
        for case in cases:
            assert call(lib, **case) == status, case


def tree(lib, parents=G, lens=G, q_start=G, B=2, T=5, words=1, mask=G, positions=G, ws=G):
    return lib.marlin_kv_tree(parents, lens, q_start, B, T, words, mask, positions, ws, None)


def test_tree_checks(lib):
    check(tree, lib,
          invalid=[dict(parents=None), dict(lens=None), dict(q_start=None), dict(mask=None), dict(positions=None), dict(ws=None),
                   dict(B=-1), dict(T=-1), dict(words=0), dict(words=-1)],
          misaligned=[dict(parents=G + 1), dict(lens=G + 2), dict(q_start=G + 2), dict(mask=G + 1), dict(positions=G + 2), dict(ws=G + 8)],
          ok=[dict(B=0), dict(T=0), dict(T=0, parents=None)])


def attention(lib, q=G, heads=4, hkv=2, D=128, page=16, B=3, T=5, max_q=2, mask=G, words=1, scale=0.1, window=0, out=G, ws=G,
              strides=(512, 128)):
    return lib.marlin_kv_tree_attention(q, *strides, heads, G, 4, hkv, D, page, G, 8, G, G, B, T, max_q, mask, words, scale, window,
                                        out, ws, 0, None)


def test_tree_attention_checks(lib):
    check(attention, lib,
          invalid=[dict(mask=None), dict(words=0), dict(words=-3), dict(heads=3), dict(hkv=0), dict(window=-1), dict(max_q=-1),
                   dict(scale=float("nan")), dict(q=None), dict(out=None), dict(ws=None), dict(T=0, words=0)],
          unsupported=[dict(D=80), dict(page=40)],
          misaligned=[dict(mask=G + 2), dict(q=G + 8), dict(out=G + 4), dict(strides=(512, 124))],
          ok=[dict(B=0), dict(T=0), dict(T=0, mask=None)])


def rope(lib, q=G, k=G, v=G, heads=4, positions=G, axes=1, table=G, rows=9, rot=128, axis=None, out=G, hkv=2, D=128, page=16, B=2,
         T=5, ws=G, strides=(1024, 128), out_strides=(512, 128), cache=G):
    axis = None if axis is None else bytes(axis)
    return lib.marlin_kv_rope_append(q, *strides, heads, k, *strides, v, *strides, positions, axes, table, rows, rot, 0, axis, out,
                                     *out_strides, cache, 4, hkv, D, page, G, 8, G, G, B, T, ws, None)


def test_rope_checks(lib):
    check(rope, lib,
          invalid=[dict(q=None), dict(k=None), dict(v=None), dict(positions=None), dict(table=None), dict(out=None), dict(ws=None),
                   dict(cache=None), dict(heads=0), dict(axes=0), dict(rows=0), dict(rot=0), dict(rot=-16), dict(rot=144),
                   dict(axes=2), dict(axes=2, axis=[0] * 63 + [2]), dict(B=-1), dict(axis=[1] + [0] * 63)],
          unsupported=[dict(rot=40), dict(rot=8), dict(D=64, rot=12), dict(axes=5, axis=[4] * 64), dict(D=96, rot=96), dict(page=8)],
          misaligned=[dict(q=G + 8), dict(k=G + 2), dict(v=G + 4), dict(positions=G + 2), dict(table=G + 8), dict(out=G + 8),
                      dict(strides=(1020, 128)), dict(out_strides=(512, -128)), dict(ws=G + 4)],
          ok=[dict(B=0), dict(T=0), dict(T=0, axes=3, axis=[0, 1, 2, 2] * 16), dict(T=0, D=64, rot=8)])


def pointers(*at):
    return (ctypes.c_void_p * len(at))(*at)


FAR = (G, G + (1 << 24), G + (2 << 24))


def compact(lib, caches=FAR, count=None, n_pages=4, hkv=2, D=128, page=16, table=G, into=None, into_pages=0, lens=G, q_start=G,
            index=G, kept=G, new=G, B=2, T=5, max_q=3, ws=G, max_pages=8):
    at = None if caches is None else pointers(*caches)
    return lib.marlin_kv_compact(at, len(caches or ()) if count is None else count, n_pages, hkv, D, page, table, max_pages, into,
                                 into_pages, lens, q_start, index, kept, new, B, T, max_q, ws, None)


def test_compact_checks(lib):
    size = 4 * 2 * 16 * 136
    check(compact, lib,
          invalid=[dict(caches=None), dict(count=0), dict(count=-1), dict(caches=(G, None)), dict(caches=(G, G)),
                   dict(caches=(G, G + (1 << 24), G + size - 16)), dict(caches=(G + size - 16, G)), dict(table=None), dict(lens=None),
                   dict(q_start=None), dict(index=None), dict(kept=None), dict(new=None), dict(ws=None), dict(B=-1), dict(T=-1),
                   dict(max_q=-1), dict(into=G), dict(into=G, into_pages=-2), dict(n_pages=0), dict(T=0, kept=None)],
          unsupported=[dict(D=32), dict(page=24), dict(into=G, into_pages=(1 << 26) + 1)],
          misaligned=[dict(caches=(G, G + (1 << 24) + 8)), dict(index=G + 2), dict(kept=G + 1), dict(new=G + 2), dict(into=G + 2, into_pages=1),
                      dict(lens=G + 1), dict(table=G + 2), dict(ws=G + 4), dict(T=0, lens=G + 1)],
          ok=[dict(B=0), dict(B=0, T=0), dict(B=0, caches=(G, G + size))])


def test_caches_that_overlap_in_any_order(lib):
    """Refused wherever the two stand; any order of caches that touch is taken.  (No requests: nothing is launched.)"""
    import random
    from w4a16_mixed_precision_gb300 import _binding as b
    size, rng = 4 * 2 * 16 * 136, random.Random(3)
    for n in (2, 3, 7, 40, 129):
        for _ in range(30):
            at = [G + size * i for i in range(n)]
            order = rng.choice([at, at[::-1], rng.sample(at, n)])
            assert compact(lib, caches=order, B=0) == b.OK
            i, j = rng.sample(range(n), 2)
            bad = list(order)
            bad[i] = bad[j] + rng.choice([0, 16, -16, size - 16, 16 - size])
            if bad[i] > 0:
                assert compact(lib, caches=bad, B=0) == b.ERR_INVALID_ARG


def copy(lib, caches=FAR, count=None, n_pages=4, hkv=2, D=128, page=16, src=G, dst=G, pairs=1, ws=G):
    at = None if caches is None else pointers(*caches)
    return lib.marlin_kv_copy_pages(at, len(caches or ()) if count is None else count, n_pages, hkv, D, page, src, dst, pairs, ws, None)


def test_copy_checks(lib):
    check(copy, lib,
          invalid=[dict(caches=None), dict(count=0), dict(caches=(G, None)), dict(caches=(G, G)), dict(src=None), dict(dst=None),
                   dict(ws=None), dict(pairs=-1), dict(n_pages=0), dict(hkv=0)],
          unsupported=[dict(D=32), dict(page=24)],
          misaligned=[dict(caches=(G + 8,)), dict(src=G + 2), dict(dst=G + 1), dict(ws=G + 8)],
          ok=[dict(pairs=0), dict(pairs=0, src=None)])


def test_pages_are_held_and_free_again():
    from w4a16_mixed_precision_gb300 import Kv4Pages
    pool = Kv4Pages(10, 16)
    a = pool.take(3)
    assert len(set(a)) == 3 and pool.free_pages == 7
    b, copies = pool.fork(a, 40)                     # two full pages and half of the third
    assert b[:2] == a[:2] and b[2] not in a and copies == [(a[2], b[2])] and pool.free_pages == 6
    assert pool.shared(a[0]) and not pool.shared(a[2])
    c, copies = pool.fork(a, 32)                     # whole pages alone
    assert c == a[:2] and copies == [] and pool.free_pages == 6
    d, copies = pool.fork(a, 0)
    assert d == [] and copies == []
    pool.free(a)
    assert pool.free_pages == 7                      # the third page alone: two forks hold the others
    pool.free(c)
    pool.free(b)
    assert pool.free_pages == 10
    for bad in (lambda: pool.take(11), lambda: pool.take(-1), lambda: pool.free([a[0]]), lambda: pool.fork(a, 16),
                lambda: pool.free([10]), lambda: pool.free([-1])):
        with pytest.raises(ValueError):
            bad()
    e = pool.take(2)
    for bad in (lambda: pool.fork(e, 33), lambda: pool.fork(e, -1), lambda: pool.free([e[0], e[0]])):
        with pytest.raises(ValueError):
            bad()
    assert pool.free_pages == 8 and not pool.shared(e[0])
    full = Kv4Pages(1, 16)
    one = full.take(1)
    with pytest.raises(ValueError):
        full.fork(one, 5)                            # no page left for the copy
    assert not full.shared(one[0])


def test_pages_against_a_model():
    """Random requests: a page is free exactly when no request lists it."""
    from w4a16_mixed_precision_gb300 import Kv4Pages
    rng, pool, held = random.Random(5), Kv4Pages(40, 16), []
    for _ in range(2000):
        what = rng.random()
        if what < 0.35 and pool.free_pages:
            n = rng.randint(1, min(5, pool.free_pages))
            held.append((pool.take(n), 16 * n - rng.randint(0, 15)))
        elif what < 0.7 and held and pool.free_pages:
            pages, length = rng.choice(held)
            length = rng.randint(0, length)
            held.append((pool.fork(pages, length)[0], length))
        elif held:
            pool.free(held.pop(rng.randrange(len(held)))[0])
        count = {}
        for pages, _ in held:
            assert len(set(pages)) == len(pages)
            for p in pages:
                count[p] = count.get(p, 0) + 1
        assert pool.free_pages == 40 - len(count)
        assert all(pool.shared(p) == (n > 1) for p, n in count.items())
