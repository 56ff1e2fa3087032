"""Numbers that the C types do not hold, given to the attention's and the verification's Python entry points: refused in
the package's manner, not as an error of the packing and not cut to their low bits (no GPU needed)."""
import ctypes
import types

import pytest

FAR = 1 << 44


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


class Memory:
    """What the wrappers ask of a device tensor, with no memory behind it."""

    is_cuda = True

    def __init__(self, torch, shape, dtype, at):
        self.shape, self.dtype, self.at = torch.Size(shape), dtype, at

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def _cache(r, torch, page=16, width=64):
    c = r.seed_cache(2, 2, 64, r.SEED_BF16, page, width, 4, page * 128, 128, 64, 16 * FAR, 32 * FAR, 48 * FAR)
    return types.SimpleNamespace(c=c, ref=ctypes.byref(c), device=0, dtype=torch.bfloat16, need={})


@pytest.mark.parametrize("how", [dict(max_length=1 << 31), dict(max_length=(1 << 32) + 64), dict(window=1 << 40), dict(max_tokens=-(1 << 33)),
                                 dict(scale="a"), dict(window=1.5)])
def test_attention(how):
    r = _lib()
    torch, _ = r._io()
    cache = _cache(r, torch)
    q, o = (Memory(torch, (2, 4, 64), torch.bfloat16, at) for at in (FAR, 2 * FAR))
    lengths = Memory(torch, (2,), torch.int32, 3 * FAR)
    with pytest.raises(ValueError):
        r.seed_decode_attend(cache, lengths, q, o, **how)
    if "scale" not in how:
        assert r.seed_attend_workspace_bytes(cache, 2, 4, **how) == 0


def test_a_table_beyond_32_bits():
    r = _lib()
    torch, _ = r._io()
    cache = _cache(r, torch, page=1 << 20, width=1 << 12)
    q, o = (Memory(torch, (2, 4, 64), torch.bfloat16, at) for at in (FAR, 2 * FAR))
    with pytest.raises(ValueError):
        r.seed_decode_attend(cache, Memory(torch, (2,), torch.int32, 3 * FAR), q, o)
    assert r.seed_attend_workspace_bytes(cache, 2, 4) == 0


def test_workspace_sizes():
    r = _lib()
    torch, _ = r._io()
    cache = _cache(r, torch, width=1 << 16)
    assert r.seed_attend_workspace_bytes(cache, 2, 4) > 0
    assert r.seed_attend_workspace_bytes(cache, 2, (1 << 32) + 4) == 0 and r.seed_attend_workspace_bytes(cache, 1 << 64, 4, ragged=True) == 0
    assert r.seed_verify_workspace_bytes(2, 500000) > 0
    assert r.seed_verify_workspace_bytes((1 << 32) + 2, 500000) == 0 and r.seed_verify_workspace_bytes(2, (1 << 32) + 500000) == 0


def test_wide_rows():
    """Rows of 2^31 values."""
    r = _lib()
    torch, _ = r._io()
    p = Memory(torch, (2, 1 << 31), torch.bfloat16, FAR)
    i, f, ends = (Memory(torch, (n,), t, at) for n, t, at in ((2, torch.int32, 2 * FAR), (2, torch.float32, 3 * FAR), (3, torch.int32, 4 * FAR)))
    with pytest.raises(ValueError):
        r.seed_verify_drafts(p, i, f, f, i, i, ends)
    rotary = types.SimpleNamespace(turns=Memory(torch, (32,), torch.float64, 5 * FAR), ref=None)
    for shape in ((1, 1, 1 << 31), (1, 1 << 31, 1)):
        x = Memory(torch, shape, torch.bfloat16, FAR)
        with pytest.raises(ValueError):
            r.seed_rotate_rows(rotary, x, Memory(torch, (1,), torch.int32, 6 * FAR), x)
