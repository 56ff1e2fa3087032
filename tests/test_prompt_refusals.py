"""Host-side refusals of the prompt path (no GPU needed): malformed calls return their status, or
raise, before anything is launched. Pointers here are never dereferenced."""
import ctypes

import pytest

BASE = 1 << 20  # a made-up, well aligned address


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


def _prefill_conv(r, conv=None, tokens=10, offsets=BASE, x=BASE, xs=64, weight=BASE, bias=None, wi=None,
                  wo=BASE + (1 << 16), y=BASE + (1 << 17), ys=64):
    conv = r.make_conv(2, 64, 4) if conv is None else conv
    return r.LIB.seed_prefill_conv(ctypes.byref(conv), tokens, offsets, x, xs, weight, bias, wi, wo, y, ys, None)


def test_conv_descriptor_and_pointers():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    assert r.LIB.seed_prefill_conv(None, 1, BASE, BASE, 1, BASE, None, None, BASE, BASE, 1, None) == arg
    for conv in (r.make_conv(0, 64, 4), r.make_conv(2, 0, 4), r.make_conv(2, 64, 0), r.make_conv(2, 64, 4, 7),
                 r.seed_conv(2, 64, 4, r.SEED_BF16, 2)):
        assert _prefill_conv(r, conv) == arg
    for conv in (r.make_conv(2, 64, 5), r.make_conv(2, 64, 1), r.make_conv(2, 64, 4, r.SEED_F16)):
        assert _prefill_conv(r, conv) == un
    for bad in (dict(offsets=None), dict(x=None), dict(weight=None), dict(wo=None), dict(y=None), dict(tokens=-1),
                dict(xs=63), dict(ys=63), dict(xs=-64), dict(x=BASE + 1), dict(weight=BASE + 2), dict(offsets=BASE + 2),
                dict(bias=BASE + 1), dict(wi=BASE + 1)):
        assert _prefill_conv(r, **bad) == arg, bad
    assert _prefill_conv(r, tokens=1 << 31) in (un, arg)


def test_conv_overlaps():
    r = _lib()
    arg = r.SEED_ERR_ARG
    # x and y: the same rows, rows that meet, and column ranges of one buffer that meet
    assert _prefill_conv(r, y=BASE) == arg
    assert _prefill_conv(r, y=BASE + 128) == arg
    assert _prefill_conv(r, xs=128, ys=128, y=BASE + 64) == arg
    assert _prefill_conv(r, xs=128, ys=256, y=BASE + 128) == arg
    # windows: in place, and the new window inside x or y
    assert _prefill_conv(r, wi=BASE + (1 << 16)) == arg
    assert _prefill_conv(r, wo=BASE + 512) == arg
    assert _prefill_conv(r, wo=BASE + (1 << 17) + 64) == arg
    assert _prefill_conv(r, wi=BASE + (1 << 17) + 64) == arg


def _decode_conv(r, conv=None, active=None, x=BASE, xs=64, weight=BASE, bias=None, wi=BASE + (1 << 16),
                 wo=BASE + (1 << 16) + 4096, y=BASE + (1 << 17), ys=64):
    conv = r.make_conv(2, 64, 4) if conv is None else conv
    return r.LIB.seed_decode_conv(ctypes.byref(conv), active, x, xs, weight, bias, wi, wo, y, ys, None)


def test_decode_conv():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    for bad in (dict(x=None), dict(weight=None), dict(wi=None), dict(wo=None), dict(y=None), dict(xs=32), dict(ys=32),
                dict(y=BASE + 2), dict(wo=BASE + (1 << 16) + 2), dict(wo=BASE), dict(wo=BASE + (1 << 17)),
                dict(wi=BASE + (1 << 17)), dict(x=BASE + 1)):
        assert _decode_conv(r, **bad) == arg, bad
    assert _decode_conv(r, r.make_conv(2, 64, 6)) == un
    assert _decode_conv(r, r.make_conv(2, 64, 4, r.SEED_F16)) == un


def _scan(r, shape=None, tokens=100, offsets=BASE, key_heads=2, qs=256, ks=256, vs=512, os=512, q=BASE, k=BASE, v=BASE,
          beta=BASE, g=BASE, S0=None, S=BASE + (1 << 24), o=BASE + (1 << 22), ws=None, ws_bytes=0):
    shape = r.make_shape(r.SEED_GDN, 3, 4, 128, 128, 16, 16, r.SEED_BF16) if shape is None else shape
    p = r.seed_prompt(tokens, offsets, key_heads, qs, ks, vs, os)
    return r.LIB.seed_prefill_scan(ctypes.byref(shape), ctypes.byref(p), q, k, v, beta, g, S0, S, o, ws, ws_bytes, None)


def test_scan():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED

    def sh(kind=0, b=3, h=4, dk=128, dv=128, f=r.SEED_BF16, io=None):
        return r.make_shape(kind, b, h, dk, dv, 16, 16, f, io)

    for bad in (sh(kind=5), sh(b=0), sh(h=0), sh(dk=0), sh(dv=-1), sh(io=9)):
        assert _scan(r, bad) == arg
    for bad in (sh(dk=96), sh(dv=256), sh(io=r.SEED_F16)):
        assert _scan(r, bad, qs=4096, ks=4096, vs=4096, os=4096) == un
    for bad in (dict(tokens=-1), dict(offsets=None), dict(key_heads=0), dict(key_heads=3), dict(key_heads=-2), dict(qs=248),
                dict(ks=128), dict(vs=504), dict(os=256), dict(qs=260), dict(vs=516), dict(q=None), dict(k=None),
                dict(v=None), dict(beta=None), dict(g=None), dict(S=None), dict(o=None), dict(q=BASE + 8), dict(v=BASE + 2),
                dict(o=BASE + (1 << 22) + 8), dict(S=BASE + (1 << 24) + 4), dict(S0=BASE + 8), dict(beta=BASE + 2),
                dict(g=BASE + 1), dict(offsets=BASE + 1)):
        assert _scan(r, **bad) == arg, bad
    # outputs that meet inputs or one another
    for bad in (dict(o=BASE), dict(o=BASE + 1024), dict(S=BASE), dict(S=BASE + (1 << 22)), dict(S0=BASE + (1 << 24) + 64),
                dict(S0=BASE + (1 << 22))):
        assert _scan(r, **bad) == arg, bad
    assert _scan(r, tokens=1 << 31) in (un, arg)


def test_scan_workspace_query():
    r = _lib()
    shape = r.make_shape(r.SEED_GDN, 3, 4, 128, 128, 16, 16, r.SEED_BF16)
    assert r.seed_prefill_workspace_bytes(shape, r.seed_prompt(-1, BASE, 2, 256, 256, 512, 512)) == 0
    assert r.seed_prefill_workspace_bytes(shape, r.seed_prompt(64, BASE, 3, 256, 256, 512, 512)) == 0


def _norm(r, rows=None, x=BASE, weight=BASE, gate=None, eps=1e-6, first=0, skip=None, scale=None, total=None,
          y=BASE + (1 << 20), res=True):
    rows = r.seed_rows(10, 4, 64, r.SEED_BF16, 256, 256, 256, 256, 256) if rows is None else rows
    n = r.seed_head_norm(weight, gate, eps, first)
    q = r.seed_residual(skip, scale, total)
    return r.LIB.seed_norm_rows(ctypes.byref(rows), x, ctypes.byref(n), ctypes.byref(q) if res else None, y, None)


def test_norm_rows():
    r = _lib()
    arg, un = r.SEED_ERR_ARG, r.SEED_ERR_UNSUPPORTED
    far = BASE + (1 << 21)

    def rows(n=10, h=4, d=64, io=r.SEED_BF16, xs=256, ys=256, gs=256, ss=256, ts=256):
        return r.seed_rows(n, h, d, io, xs, ys, gs, ss, ts)

    for bad in (rows(n=-1), rows(h=0), rows(d=0), rows(io=4), rows(xs=255), rows(ys=128)):
        assert _norm(r, bad) == arg
    assert _norm(r, rows(gs=8), gate=far) == arg
    assert _norm(r, rows(ss=8), skip=far) == arg
    assert _norm(r, rows(ts=8), skip=far, total=far + (1 << 20)) == arg
    assert _norm(r, rows(io=r.SEED_F16)) == un
    assert _norm(r, rows(n=1 << 31)) == un
    for bad in (dict(x=None), dict(y=None), dict(weight=None), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(first=2), dict(scale=far), dict(x=BASE + 1), dict(gate=far + 1), dict(weight=BASE + 2),
                dict(y=BASE + 2), dict(y=BASE + 512), dict(skip=far, total=far + 64),
                dict(skip=far, total=BASE + (1 << 20)), dict(skip=far, scale=far + 2)):
        assert _norm(r, **bad) == arg, bad
    assert _norm(r, rows(n=0), x=None, y=None) == r.SEED_OK  # nothing to do


def test_wrappers_refuse_wrong_tensors():
    r = _lib()
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(4, 64)
    off = torch.zeros(3, dtype=torch.int32)
    win = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    conv = r.make_conv(2, 64, 4)
    with pytest.raises(ValueError, match="device tensor"):
        r.seed_prefill_conv(conv, x, off, w, None, win, torch.empty_like(x), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        r.seed_decode_conv(conv, x[:2], w, None, win, torch.empty_like(x[:2]), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        r.seed_norm_rows(x.view(4, 1, 64), w[:1], torch.empty_like(x).view(4, 1, 64), stream=0)
    with pytest.raises(ValueError, match="rows, heads, dim"):
        r.seed_norm_rows(x, w[:1], x, stream=0)
    with pytest.raises(ValueError, match="dtype"):
        r.seed_norm_rows(x.view(4, 1, 64).half(), w[:1], x.view(4, 1, 64).half(), stream=0)
    shape = r.make_shape(r.SEED_GDN, 2, 2, 64, 64, 16, 16, r.SEED_BF16)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    s = torch.zeros(2, 2, 64, 64)
    b = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        r.seed_prefill_scan(shape, off, q, q, q, b, b, s, q.clone(), stream=0)
    with pytest.raises(ValueError, match="key heads"):
        r.seed_prefill_scan(shape, off, q.expand(4, 2, 64)[:, :0], q, q, b, b, s, q.clone(), stream=0)
