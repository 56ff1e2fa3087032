"""Keys and values in one buffer: a cache is accepted if and only if no value of k is one of v, by a listing of all places
(no GPU needed; pointers are never dereferenced)."""
import ctypes
import random

import numpy as np
import pytest

UNIT = 8  # bf16 values of 16 bytes: strides and the way from k to v are multiples of it


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


def _places(pages, page, heads, dim, ps, ts, hs):
    """Where a pool's values lie, in units from its first."""
    p, s, h, d = np.meshgrid(np.arange(pages), np.arange(page), np.arange(heads), np.arange(dim // UNIT), indexing="ij")
    return ((p * ps + s * ts + h * hs) // UNIT + d).ravel()


def _status(r, pages, page, heads, dim, ps, ts, hs, way):
    """Of both entry points' checks, with no tokens: nothing is launched."""
    k = 1 << 44
    cache = r.seed_cache(1, heads, dim, r.SEED_BF16, page, 4, pages, ps, ts, hs, k, k + 2 * way, 1 << 40)
    none = r.seed_tokens(0, 1 << 41, 1 << 42, heads, heads * dim, heads * dim, heads * dim, heads * dim)
    how = r.seed_attend(1, 64, 0, 0.1)
    a = r.LIB.seed_cache_append(ctypes.byref(cache), ctypes.byref(none), None, None, None, None, None, None)
    b = r.LIB.seed_decode_attend(ctypes.byref(cache), ctypes.byref(none), ctypes.byref(how), None, None, None, None, 0, None)
    assert a == b
    return a


def _check(r, layout, way):
    pages, page, heads, dim, ps, ts, hs = layout
    at = _places(*layout)
    assert len(np.unique(at)) == len(at), "the layout itself overlaps"
    meet = bool(np.isin(at + way // UNIT, at).any())
    want = r.SEED_ERR_ARG if meet else r.SEED_OK
    assert _status(r, *layout, way) == want, (layout, way, meet)
    return meet


@pytest.mark.parametrize("layout,way", [
    ((4, 16, 1, 64, 1984, 128, 64), 64),        # v's last slot of a page on k's first one of the next
    ((30, 16, 1, 128, 4696, 304, 128), 152),
    ((3, 16, 1, 64, 3136, 192, 64), 3136),      # v's first page is k's second
    ((3, 16, 2, 64, 5000, 160, 2480), 80),      # [key_heads][page]: the same between heads
    ((3, 16, 2, 64, 4184, 256, 72), 8),
])
def test_pools_that_meet_are_refused(layout, way):
    assert _check(_lib(), layout, way)


@pytest.mark.parametrize("layout,way", [
    ((4, 16, 1, 64, 2048, 128, 64), 64),        # token by token, pages whole numbers of tokens apart
    ((4, 16, 1, 64, 2056, 128, 64), 64),        # and not, with room for v's last slot
    ((4, 16, 2, 64, 16 * 256, 256, 128), 64),   # head by head
    ((4, 16, 2, 64, 16 * 256, 256, 64), 128),
    ((4, 16, 1, 64, 2 * 16 * 64, 64, 64), 16 * 64),
    ((4, 16, 2, 64, 4 * 16 * 64, 64, 16 * 64), 2 * 16 * 64),
    ((4, 16, 2, 64, 4 * 16 * 64, 64, 2 * 16 * 64), 16 * 64),
    ((2, 16, 1, 64, 16 * 64, 64, 64), 2 * 16 * 64),
    ((1, 16, 1, 64, 8, 128, 8), 64),            # the strides of a single page and head count for nothing
])
def test_pools_side_by_side_are_taken(layout, way):
    assert not _check(_lib(), layout, way)


def test_any_layout():
    """Random strides, close together, both orders, v before k too."""
    r = _lib()
    rng = random.Random(5)
    met = 0
    for _ in range(4000):
        pages, page, heads, dim = rng.randint(1, 4), 16, rng.randint(1, 3), 64

        def room(least):  # a stride with a little room, or a lot of it
            return least + UNIT * rng.choice([0, 0, 1, 3, 8, 9, 16, rng.randint(0, 60)])

        if rng.random() < 0.5:
            hs = room(dim)
            ts = room((heads - 1) * hs + dim)
        else:
            ts = room(dim)
            hs = room((page - 1) * ts + dim)
        ps = room((page - 1) * ts + (heads - 1) * hs + dim)
        span = (pages - 1) * ps + (page - 1) * ts + (heads - 1) * hs + dim
        way = rng.choice([dim, hs, ts, ps, heads * hs, page * ts, hs // 2, ts // 2, ps // 2, ps + dim, ps + ts, ps - dim, rng.randint(0, span)])
        way = way // UNIT * UNIT * rng.choice([1, 1, -1])
        met += _check(r, (pages, page, heads, dim, ps, ts, hs), way)
    assert 400 < met < 3600
