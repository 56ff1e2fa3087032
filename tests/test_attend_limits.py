"""Limits of the attention's and the verification's launches and sizes (no GPU needed; pointers are never dereferenced, and
no call here launches: those within the limits have no tokens)."""
import ctypes

import pytest

FAR = 1 << 44
MOST = (1 << 32) - 1  # threads of a launch


def _lib():
    return pytest.importorskip("rank_recurrent_state_amd._lib",
                               reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")


def _attend(r, batch, key_heads, heads, max_length, max_tokens=1, dim=64, width=64):
    cache = r.seed_cache(batch, key_heads, dim, r.SEED_BF16, 16, width, 4, 16 * key_heads * dim, key_heads * dim, dim, 16 * FAR, 32 * FAR, 48 * FAR)
    none = r.seed_tokens(0, FAR, 2 * FAR, heads, heads * dim, 0, 0, heads * dim)
    how = r.seed_attend(max_tokens, max_length, 0, 0.1)
    return r.LIB.seed_decode_attend(ctypes.byref(cache), ctypes.byref(none), ctypes.byref(how), None, None, None, 3 * FAR, 1 << 40, None)


def test_attention_workgroups():
    """A workgroup per request and key head has 256 threads for up to 128 keys and 512 for up to 1024; one for each 16 rows
    of 256 is always counted."""
    r = _lib()
    ok, un = r.SEED_OK, r.SEED_ERR_UNSUPPORTED
    for key_heads in (1, 4):
        for length, threads in ((128, 256), (129, 512), (1024, 512)):
            most = MOST // threads // key_heads
            assert _attend(r, most, key_heads, key_heads, length) == ok, (key_heads, length)
            assert _attend(r, most + 1, key_heads, key_heads, length) == un, (key_heads, length)
    assert _attend(r, 1 << 20, 1, 16, 1024) == un  # rows


def test_verification_workgroups():
    """Up to 32768 tokens a request is one workgroup of 1024 threads, beyond one of 256 for 4096 tokens."""
    r = _lib()

    def call(batch, vocab):
        d = r.seed_drafts(batch, vocab, r.SEED_F32, 1, FAR, vocab, vocab)
        return r.LIB.seed_verify_drafts(ctypes.byref(d), 2 * FAR, None, 3 * FAR, 4 * FAR, 5 * FAR, 6 * FAR, 7 * FAR, 8 * FAR, 1 << 50, None)

    for batch, vocab in ((MOST // 1024 + 1, 1), (MOST // 1024 + 1, 32768), ((1 << 31) - 1, 2), (1 << 23, 32769), (1 << 22, 32768)):
        assert call(batch, vocab) == r.SEED_ERR_UNSUPPORTED, (batch, vocab)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("share,max_tokens", [(1, 1), (4, 6), (16, 32)])
def test_attention_workspace_bound(io, dim, share, max_tokens):
    """At most 2 (511 + key_heads) places of up to 64 rows, none from 512 key heads on, and 8 bytes for each request and
    row block; whatever the lengths."""
    r = _lib()
    code = {"bf16": r.SEED_BF16, "f32": r.SEED_F32}[io]
    for key_heads in (1, 2, 3, 7, 8, 100, 256, 257, 300, 510, 511, 512, 513, 1024, 4096):
        for batch in (1, 5):
            if batch * share * max_tokens * key_heads >= 1 << 24:
                continue
            for length in (4096, 1 << 20):
                cache = r.seed_cache(batch, key_heads, dim, code, 16, 1 << 16, 4, 16 * key_heads * dim, key_heads * dim, dim, 16 * FAR, 32 * FAR, 48 * FAR)
                new = r.seed_tokens(batch, FAR, 2 * FAR, share * key_heads, share * key_heads * dim, 0, 0, share * key_heads * dim)
                how = r.seed_attend(max_tokens, length, 0, 0.1)
                need = r.LIB.seed_attend_workspace_bytes(ctypes.byref(cache), ctypes.byref(new), ctypes.byref(how))
                rows = min(share * max_tokens, 64)
                notes = 8 * batch * -(-share * max_tokens // 16)
                places = 2 * (511 + key_heads) if key_heads < 512 else 0
                assert (length == 4096 or need > 0) and need <= places * rows * (dim + 2) * 4 + notes, (key_heads, batch, length)
