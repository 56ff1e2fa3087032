"""Host-side checks of the attention layers' entry points and of draft verification (no GPU needed):
malformed calls return their status, or raise, before anything is launched; size queries; the rotary
tables. Pointers here are never dereferenced."""
import ctypes

import numpy as np
import pytest

import attend_ref as ref

BASE = 1 << 20  # a made-up, well aligned address
FAR = 1 << 40
INF, NAN = float("inf"), float("nan")


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


# ---- rotary tables --------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [2, 6, 64, 128, 256])
@pytest.mark.parametrize("how", [dict(kind="plain"), dict(kind="plain", base=500000.0), dict(kind="linear", factor=4.0),
                                 dict(kind="base", factor=8.0), dict(kind="parts", factor=8.0, length=8192.0, low=1.0, high=4.0),
                                 dict(kind="parts", factor=32.0, length=4096.0), dict(kind="index", factor=16.0, length=4096.0)])
def test_turns(dim, how):
    r = _lib()
    if how["kind"] == "index" and dim < 64:
        pytest.skip("no room for a ramp: test_turns_step")
    kinds = dict(plain=r.SEED_ROTARY_PLAIN, linear=r.SEED_ROTARY_LINEAR, base=r.SEED_ROTARY_BASE, parts=r.SEED_ROTARY_PARTS,
                 index=r.SEED_ROTARY_INDEX)
    args = {k: v for k, v in how.items() if k != "kind"}
    got = r.seed_rotary_turns(dim, scaling=kinds[how["kind"]], **args)
    # a few operations of 2^-53 each, powers and logarithms among them
    np.testing.assert_allclose(got, ref.turns(dim, **how), rtol=1e-13)


def test_turns_step():
    """Where the ramp's ends meet, pairs up to it stay and those behind stretch."""
    r = _lib()
    plain = np.array(r.seed_rotary_turns(4, base=100.0))
    got = np.array(r.seed_rotary_turns(4, base=100.0, scaling=r.SEED_ROTARY_INDEX, factor=10.0, length=1.0, low=30.0, high=31.0))
    np.testing.assert_allclose(got, plain * [1.0, 0.1], rtol=1e-15)


def test_turns_refusals():
    r = _lib()

    def call(kind=0, base=1e4, factor=2.0, length=100.0, low=1.0, high=4.0, dim=8):
        out = (ctypes.c_double * 64)()
        how = r.seed_rotary_scaling(kind, base, factor, length, low, high)
        return r.LIB.seed_rotary_turns(ctypes.byref(how), dim, out)

    assert r.LIB.seed_rotary_turns(None, 8, (ctypes.c_double * 4)()) == r.SEED_ERR_ARG
    assert r.LIB.seed_rotary_turns(ctypes.byref(r.seed_rotary_scaling(0, 1e4)), 8, None) == r.SEED_ERR_ARG
    for bad in (dict(kind=-1), dict(kind=5), dict(base=0.0), dict(base=-1.0), dict(base=INF), dict(base=NAN), dict(dim=7), dict(dim=0),
                dict(dim=-2), dict(kind=1, factor=0.0), dict(kind=1, factor=NAN), dict(kind=2, factor=INF), dict(kind=3, length=0.0),
                dict(kind=3, low=0.0), dict(kind=3, low=4.0), dict(kind=3, high=INF), dict(kind=4, base=1.0), dict(kind=4, length=NAN)):
        assert call(**bad) == r.SEED_ERR_ARG, bad
    assert call(factor=0.0, length=-1.0, low=9.0, high=1.0) == r.SEED_OK  # ignored by a plain table
    assert call(kind=1, length=-1.0, low=9.0, high=1.0) == r.SEED_OK
    # turns beyond fp64
    assert call(kind=1, factor=5e-324) == r.SEED_ERR_ARG and call(kind=2, factor=1e-300, dim=4) == r.SEED_ERR_ARG


def _rotary(r, dim=64, interleaved=0, amplitude=1.0, turns=5 * FAR):
    return r.seed_rotary(dim, interleaved, amplitude, turns)


def test_rotate_rows():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED

    def call(n=10, h=4, d=64, io=r.SEED_BF16, xs=256, ys=256, rotary=None, x=BASE, positions=4 * FAR, y=FAR):
        rows = r.seed_rows(n, h, d, io, xs, ys)
        rot = _rotary(r) if rotary is None else rotary
        return r.LIB.seed_rotate_rows(ctypes.byref(rows), ctypes.byref(rot), x, positions, y, None)

    assert r.LIB.seed_rotate_rows(None, ctypes.byref(_rotary(r)), BASE, BASE, BASE, None) == arg
    assert r.LIB.seed_rotate_rows(ctypes.byref(r.seed_rows(1, 1, 64, 1, 64, 64)), None, BASE, FAR, BASE, None) == arg
    for bad in (dict(n=-1), dict(h=0), dict(d=0), dict(io=7), dict(xs=255), dict(ys=10), dict(x=None), dict(y=None),
                dict(positions=None), dict(x=BASE + 1), dict(y=FAR + 1), dict(positions=4 * FAR + 2),
                dict(rotary=_rotary(r, 66)), dict(rotary=_rotary(r, 7)), dict(rotary=_rotary(r, 0)), dict(rotary=_rotary(r, -2)),
                dict(rotary=_rotary(r, interleaved=2)), dict(rotary=_rotary(r, amplitude=INF)), dict(rotary=_rotary(r, amplitude=NAN)),
                dict(rotary=_rotary(r, turns=None)), dict(rotary=_rotary(r, turns=FAR + 4)),
                # overlaps: shifted rows, rows of another stride, positions and turns inside y
                dict(y=BASE + 128), dict(xs=512, y=BASE), dict(positions=FAR + 16), dict(rotary=_rotary(r, turns=FAR + 512))):
        assert call(**bad) == arg, bad
    assert call(io=r.SEED_F16) == un
    assert call(n=1 << 31) == un
    assert call(n=(1 << 31) - 1, xs=1 << 40, ys=1 << 40, y=BASE) == un
    assert call(n=0, x=None, y=None, positions=None) == r.SEED_OK


# ---- the cache ------------------------------------------------------------------------------------

def _cache(r, batch=3, kh=2, dim=128, io=None, page=16, width=8, pages=30, ps=None, ts=256, hs=128, k=16 * FAR, v=32 * FAR, table=8 * FAR):
    return r.seed_cache(batch, kh, dim, r.SEED_BF16 if io is None else io, page, width, pages, 16 * 256 if ps is None else ps, ts,
                        hs, k, v, table)


def _tokens(r, n=5, offsets=2 * FAR, lengths=3 * FAR, heads=4, qs=512, ks=256, vs=256, os=512):
    return r.seed_tokens(n, offsets, lengths, heads, qs, ks, vs, os)


def _append(r, cache=None, tokens=None, rotary=None, q=BASE, k=BASE + (1 << 16), v=BASE + (1 << 17), out=FAR):
    cache = _cache(r) if cache is None else cache
    tokens = _tokens(r) if tokens is None else tokens
    return r.LIB.seed_cache_append(ctypes.byref(cache), ctypes.byref(tokens), None if rotary is None else ctypes.byref(rotary),
                                   q, k, v, out, None)


def _attend(r, cache=None, tokens=None, most=1, length=128, window=0, scale=0.1, q=BASE, o=FAR, lse=None, ws=6 * FAR, size=1 << 40):
    cache = _cache(r) if cache is None else cache
    tokens = _tokens(r) if tokens is None else tokens
    how = r.seed_attend(most, length, window, scale)
    return r.LIB.seed_decode_attend(ctypes.byref(cache), ctypes.byref(tokens), ctypes.byref(how), q, o, lse, ws, size, None)


def test_cache_descriptor():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    how = r.seed_attend(1, 128, 0, 0.1)
    assert r.LIB.seed_cache_append(None, ctypes.byref(_tokens(r)), None, None, BASE, BASE, None, None) == arg
    assert r.LIB.seed_cache_append(ctypes.byref(_cache(r)), None, None, None, BASE, BASE, None, None) == arg
    assert r.LIB.seed_decode_attend(None, ctypes.byref(_tokens(r)), ctypes.byref(how), BASE, FAR, None, None, 0, None) == arg
    assert r.LIB.seed_decode_attend(ctypes.byref(_cache(r)), ctypes.byref(_tokens(r)), None, BASE, FAR, None, None, 0, None) == arg
    for call in (_append, _attend):
        for bad in (dict(batch=0), dict(kh=0), dict(dim=0), dict(page=0), dict(width=0), dict(pages=0), dict(io=5), dict(k=None),
                    dict(v=None), dict(table=None), dict(k=16 * FAR + 8), dict(v=32 * FAR + 2), dict(table=8 * FAR + 2), dict(ts=0),
                    dict(hs=-128), dict(ps=4100), dict(ts=260), dict(hs=132),
                    # heads, tokens or pages that overlap, and strides in neither order
                    dict(hs=120), dict(ts=128), dict(ps=4096 - 8), dict(ts=136, hs=128), dict(ts=128, hs=15 * 128)):
            assert call(r, _cache(r, **bad)) == arg, bad
        for bad in (dict(dim=96), dict(dim=512), dict(io=r.SEED_F16), dict(page=8), dict(page=24), dict(page=1 << 21),
                    dict(page=1 << 20, width=1025, ps=1 << 40), dict(kh=1 << 30, hs=1 << 40), dict(pages=1 << 40, ps=1 << 40)):
            assert call(r, _cache(r, **bad)) == un, bad
        # keys and values that share bytes: the same pages, half a page on, a head inside
        for v in (16 * FAR, 16 * FAR + 4096, 16 * FAR + 256, 16 * FAR + 8192 * 29):
            assert call(r, _cache(r, v=v)) == arg, v


def test_cache_layouts_side_by_side():
    """Keys and values in one buffer, by pages, tokens or heads: accepted up to the next check (tokens 0)."""
    r = _lib()
    none = _tokens(r, n=0)
    k = 16 * FAR
    for cache in (_cache(r, ps=2 * 4096, v=k + 2 * 4096), _cache(r, ps=2 * 4096, ts=512, v=k + 2 * 256),
                  _cache(r, ps=2 * 4096, ts=512, hs=256, v=k + 2 * 128), _cache(r, ps=4096, ts=128, hs=16 * 128),
                  _cache(r, ps=8192, ts=256, hs=32 * 128, v=k + 2 * 128), _cache(r, kh=1, hs=8, ts=128, ps=2048),
                  _cache(r, pages=1, ps=8)):
        assert _append(r, cache, none, q=None, out=None) == r.SEED_OK
        assert _attend(r, cache, none) == r.SEED_OK
        cache.v = cache.k + 2 * 64
        assert _append(r, cache, none, q=None, out=None) == r.SEED_ERR_ARG


def test_append():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    for bad in (dict(n=-1), dict(lengths=None), dict(n=4, offsets=None), dict(heads=0), dict(heads=3), dict(heads=-2), dict(qs=511),
                dict(ks=255), dict(vs=0), dict(os=8), dict(offsets=2 * FAR + 2), dict(lengths=3 * FAR + 1)):
        assert _append(r, tokens=_tokens(r, **bad)) == arg, bad
    assert _append(r, tokens=_tokens(r, n=1 << 31)) == un
    assert _append(r, tokens=_tokens(r, n=(1 << 31) - 1, qs=1 << 40)) == un
    for bad in (dict(k=None), dict(v=None), dict(out=None), dict(q=None), dict(q=BASE + 1), dict(k=BASE + 1), dict(v=BASE + 1),
                dict(out=FAR + 1), dict(rotary=_rotary(r, 130)), dict(rotary=_rotary(r, 3)), dict(rotary=_rotary(r, amplitude=NAN)),
                # q_out over the keys, shifted over q, over offsets, lengths, the table, the turns or a pool
                dict(out=BASE + (1 << 16)), dict(out=BASE + 256), dict(out=2 * FAR), dict(out=3 * FAR), dict(out=8 * FAR),
                dict(out=5 * FAR, rotary=_rotary(r)), dict(out=16 * FAR + 4096), dict(k=32 * FAR), dict(q=16 * FAR),
                dict(rotary=_rotary(r, turns=32 * FAR))):
        assert _append(r, **bad) == arg, bad
    assert _append(r, tokens=_tokens(r, n=0, heads=0), q=None, out=None, k=None, v=None) == r.SEED_OK


def test_attend():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    for bad in (dict(n=-1), dict(lengths=None), dict(n=4, offsets=None), dict(heads=0), dict(heads=5), dict(qs=504), dict(os=504),
                dict(qs=516), dict(os=516)):
        assert _attend(r, tokens=_tokens(r, **bad)) == arg, bad
    for bad in (dict(most=0), dict(most=-1), dict(length=0), dict(length=129), dict(window=-1), dict(scale=INF), dict(scale=NAN),
                dict(scale=3e38), dict(scale=0.0), dict(q=None), dict(o=None), dict(q=BASE + 8), dict(o=FAR + 2), dict(lse=FAR + (1 << 20) + 2),
                # overlaps
                dict(o=BASE), dict(o=BASE + 1024), dict(lse=FAR + 64), dict(o=16 * FAR), dict(lse=32 * FAR + 64), dict(o=8 * FAR),
                dict(o=2 * FAR), dict(lse=3 * FAR), dict(lse=BASE + 8)):
        assert _attend(r, **bad) == arg, bad
    assert _attend(r, most=33) == un
    assert _attend(r, _cache(r, batch=1 << 24), _tokens(r, n=1 << 24)) == un
    assert _attend(r, tokens=_tokens(r, n=1 << 31)) == un
    assert _attend(r, tokens=_tokens(r, n=0), q=None, o=None, ws=None, size=0) == r.SEED_OK


def test_attend_workspace():
    r = _lib()
    long = _cache(r, batch=1, page=1 << 10, width=1 << 8, ps=(1 << 10) * 256, pages=300)
    one = _tokens(r, n=1, offsets=None)
    how = r.seed_attend(1, 1 << 18, 0, 0.1)
    need = r.LIB.seed_attend_workspace_bytes(ctypes.byref(long), ctypes.byref(one), ctypes.byref(how))
    assert 0 < need < 1 << 28  # does not grow with the cache
    for bad in (dict(ws=None), dict(size=need - 1), dict(ws=None, size=need)):
        assert _attend(r, long, one, length=1 << 18, **bad) == r.SEED_ERR_WORKSPACE, bad
    for ws in (6 * FAR + 4, BASE, FAR + 16, 16 * FAR, 8 * FAR - 64):
        assert _attend(r, long, one, length=1 << 18, ws=ws, size=need) == r.SEED_ERR_ARG, ws
    how.max_length = 64  # one workgroup's keys
    assert r.LIB.seed_attend_workspace_bytes(ctypes.byref(long), ctypes.byref(one), ctypes.byref(how)) == 0
    how.max_length = 0
    assert r.LIB.seed_attend_workspace_bytes(ctypes.byref(long), ctypes.byref(one), ctypes.byref(how)) == 0
    assert r.LIB.seed_attend_workspace_bytes(None, None, None) == 0


# ---- verification ---------------------------------------------------------------------------------

def _verify(r, batch=3, vocab=500000, io=None, n=8, offsets=2 * FAR, tstride=500000, dstride=500000, target=BASE, draft=4 * FAR,
            drafts=5 * FAR, uniforms=6 * FAR, draws=7 * FAR, out=8 * FAR, counts=9 * FAR, ws=10 * FAR, size=1 << 30):
    d = r.seed_drafts(batch, vocab, r.SEED_F32 if io is None else io, n, offsets, tstride, dstride)
    return r.LIB.seed_verify_drafts(ctypes.byref(d), target, draft, drafts, uniforms, draws, out, counts, ws, size, None)


def test_verify():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    assert r.LIB.seed_verify_drafts(None, *[BASE] * 8, 0, None) == arg
    for bad in (dict(batch=0), dict(vocab=0), dict(n=-1), dict(io=9), dict(offsets=None), dict(tstride=499999), dict(dstride=499999),
                dict(target=None), dict(drafts=None), dict(uniforms=None), dict(draws=None), dict(out=None), dict(counts=None),
                dict(target=BASE + 2), dict(draft=4 * FAR + 1), dict(offsets=2 * FAR + 2), dict(drafts=5 * FAR + 1), dict(out=8 * FAR + 2),
                dict(counts=9 * FAR + 3), dict(ws=10 * FAR + 8),
                # overlaps: out shifted over drafts or over any other input, counts over drafts, the workspace over anything
                dict(out=5 * FAR + 4), dict(out=BASE), dict(out=6 * FAR), dict(out=7 * FAR), dict(counts=5 * FAR), dict(counts=8 * FAR),
                dict(ws=5 * FAR), dict(ws=8 * FAR), dict(ws=BASE)):
        assert _verify(r, **bad) == arg, bad
    assert _verify(r, io=r.SEED_F16) == un
    assert _verify(r, n=1 << 31) == un
    assert _verify(r, batch=1 << 20, vocab=1 << 20) == un
    assert _verify(r, n=(1 << 31) - 1, tstride=1 << 40) == un
    need = r.seed_verify_workspace_bytes(3, 500000)
    assert need > 0 and r.seed_verify_workspace_bytes(3, 1000) == 0  # small ones are done in one launch
    for bad in (dict(ws=None), dict(size=need - 1)):
        assert _verify(r, **bad) == r.SEED_ERR_WORKSPACE
    assert r.seed_verify_workspace_bytes(0, 500000) == 0


def test_wrappers_refuse_wrong_tensors():
    r = _lib()
    import torch
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        r.Cache(k, k.clone(), table)
    with pytest.raises(ValueError, match="page, key_heads, dim"):
        r.Cache(k[0], k[0], table)
    with pytest.raises(ValueError, match="dtype"):
        r.Cache(k, k.float(), table)
    with pytest.raises(ValueError, match="int32"):
        r.Cache(k, k.clone(), table.long())
    with pytest.raises(ValueError, match="float64"):
        r.Rotary(torch.zeros(4))
    with pytest.raises(r.SeedError):
        r.make_rotary(7, device="cpu")
    p = torch.zeros(4, 100)
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="device tensor"):
        r.seed_verify_drafts(p, i, f, f, i.clone(), i.clone(), i, stream=0)
    with pytest.raises(ValueError, match="rows, vocab"):
        r.seed_verify_drafts(p[0], i, f, f, i.clone(), i.clone(), i, stream=0)
    with pytest.raises(ValueError, match="dtype"):
        r.seed_verify_drafts(p.half(), i, f, f, i.clone(), i.clone(), i, stream=0)
