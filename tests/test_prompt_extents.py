"""Host-side refusals of the prompt path's calls whose buffers could not lie in an address range (no GPU
needed): sizes and strides that are each within their limits and whose products pass 64 bits. Pointers
here are never dereferenced."""
import ctypes

import pytest

BASE, FAR = 1 << 20, 1 << 40  # made-up, well aligned addresses
MOST, STRIDE = (1 << 31) - 1, 1 << 40


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


@pytest.mark.parametrize("io", ["SEED_F32", "SEED_BF16"])
def test_convolutions(io):
    r = _lib()
    un = r.SEED_ERR_UNSUPPORTED

    def prefill(batch, channels, tokens, xs, ys, x=BASE, y=FAR):
        c = r.make_conv(batch, channels, 4, getattr(r, io))
        return r.LIB.seed_prefill_conv(ctypes.byref(c), tokens, BASE, x, xs, BASE, None, None, 2 * FAR, y, ys, None)

    def decode(batch, channels, xs, ys, x=BASE, y=FAR):
        c = r.make_conv(batch, channels, 4, getattr(r, io))
        return r.LIB.seed_decode_conv(ctypes.byref(c), None, x, xs, BASE, None, 2 * FAR, 3 * FAR, y, ys, None)

    assert prefill(2, 64, MOST, STRIDE, STRIDE, y=BASE) == un  # in place, whatever the wrapped ends say
    assert prefill(2, 64, MOST, STRIDE, 64) == un
    assert prefill(2, 64, MOST, 64, STRIDE) == un
    assert prefill(MOST, MOST, 1, MOST, MOST) == un  # the windows
    assert decode(MOST, 64, STRIDE, STRIDE, y=BASE) == un
    assert decode(MOST, 64, 64, STRIDE) == un
    assert decode(MOST, 1 << 28, 1 << 28, 1 << 28) == un
    # an end that passes the last address
    assert prefill(2, 64, 1 << 20, 64, 64, x=(1 << 64) - (1 << 20)) == un


@pytest.mark.parametrize("io", ["SEED_F32", "SEED_BF16"])
def test_scan(io):
    r = _lib()

    def scan(kind, heads, tokens, stride, o=FAR):
        s = r.make_shape(kind, 1, heads, 128, 128, 16, 16, r.SEED_BF16, getattr(r, io))
        p = r.seed_prompt(tokens, BASE, 1, stride, stride, stride, stride)
        return r.LIB.seed_prefill_scan(ctypes.byref(s), ctypes.byref(p), BASE, BASE, BASE, BASE, BASE, None, 2 * FAR, o, 3 * FAR,
                                       1 << 50, None)

    for kind in (r.SEED_GDN, r.SEED_KDA, r.SEED_MAMBA2):
        assert scan(kind, 4, MOST, STRIDE, o=BASE) == r.SEED_ERR_UNSUPPORTED
        assert scan(kind, 1 << 30, MOST, 1 << 37) == r.SEED_ERR_UNSUPPORTED  # beta and g too


@pytest.mark.parametrize("io", ["SEED_F32", "SEED_BF16"])
def test_norm(io):
    r = _lib()

    def norm(n, strides, heads=4, dim=64, gate=None, y=FAR):
        q = r.seed_rows(n, heads, dim, getattr(r, io), *strides)
        m = r.seed_head_norm(BASE, gate, 1e-6, 0)
        return r.LIB.seed_norm_rows(ctypes.byref(q), BASE, ctypes.byref(m), None, y, None)

    un = r.SEED_ERR_UNSUPPORTED
    assert norm(MOST, (STRIDE, STRIDE - 64, 0, 0, 0), y=BASE) == un
    assert norm(MOST, (STRIDE, 256, 0, 0, 0)) == un
    assert norm(MOST, (256, 256, STRIDE, 0, 0), gate=FAR) == un
    # strides of absent buffers are not looked at, whatever they hold
    big = (1 << 63) - 1
    assert norm(10, (256, 256, big, big, -big), y=BASE) == r.SEED_ERR_ARG  # y over x, but the weight at the same address
