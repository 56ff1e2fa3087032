"""Which prompts of the chunked scan are cut into segments, seen by the workspace that they need (no GPU
needed): those that were measured to gain by it, and none that were measured to lose."""
import pytest


def _cut(kind, batch, heads, dk, dv, length, io="SEED_BF16"):
    r = pytest.importorskip("rank_recurrent_state_amd._lib",
                            reason="libseed.so not built (python -m rank_recurrent_state_amd.build)")
    shape = r.make_shape(getattr(r, kind), batch, heads, dk, dv, 16, 16, r.SEED_BF16, getattr(r, io))
    p = r.seed_prompt(batch * length, None, heads, heads * dk, heads * dk, heads * dv, heads * dv)
    return r.seed_prefill_workspace_bytes(shape, p) > 0


@pytest.mark.parametrize("units", [(1, 176), (1, 192), (1, 224), (4, 64), (1, 256)])
@pytest.mark.parametrize("dk", [64, 128])
def test_three_segments_of_mamba2_with_64_columns(units, dk):
    assert not _cut("SEED_MAMBA2", *units, dk, 64, 1024)
    assert not _cut("SEED_MAMBA2", *units, dk, 64, 2048)
    assert _cut("SEED_MAMBA2", *units, dk, 64, 8192)


def test_prompts_that_gain():
    for units in (16, 64, 128, 170):
        for n in (1024, 2048, 8192):
            assert _cut("SEED_MAMBA2", 1, units, 128, 64, n)
    for units in (16, 64, 85, 128):
        for n in (1024, 2048, 8192):
            assert _cut("SEED_MAMBA2", 1, units, 128, 128, n)
    for units in (8, 16, 32, 64, 85):
        for n in (2048, 8192):
            assert _cut("SEED_GDN", 1, units, 128, 128, n)
    assert _cut("SEED_GDN", 1, 32, 128, 128, 1024)


def test_prompts_that_lose():
    for kind, dv in (("SEED_GDN", 128), ("SEED_MAMBA2", 64)):
        for units in (16, 64, 128):
            assert not _cut(kind, 1, units, 128, dv, 512)
    for n in (1024, 2048, 8192):
        assert not _cut("SEED_GDN", 1, 128, 128, 128, n)
    assert not _cut("SEED_GDN", 1, 64, 128, 128, 1024) and not _cut("SEED_GDN", 1, 85, 128, 128, 1024)
    assert not _cut("SEED_GDN", 1, 16, 128, 128, 8192, "SEED_F32") and not _cut("SEED_KDA", 1, 16, 128, 128, 8192)
