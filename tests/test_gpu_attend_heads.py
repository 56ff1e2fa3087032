"""GPU test of the attention over more key heads than a call has workgroups for one each: every workgroup has a key head's
turns whole, and the workspace holds no partial results."""
from __future__ import annotations

import pytest

import test_gpu_attend as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kh,share,new", [(511, 1, [1, 1]), (512, 1, [1, 1]), (520, 2, [3, 1]), (515, 5, [4, 2])])
def test_many_key_heads(dtype, kh, share, new):
    rrs, torch = base._rrs()
    lengths = [1100, 37]
    cache = base._cache(rrs, torch, lengths, kh, 64, 16, dtype, kh)
    cache = rrs.Cache(cache.k, cache.v, torch.nn.functional.pad(cache.table, (0, 4096 - cache.table.shape[1]), value=-1))  # a far limit
    n, heads, most = sum(new), kh * share, max(new)
    need = rrs.seed_attend_workspace_bytes(cache, n, heads, max_tokens=most, ragged=True)
    blocks = 1 if most * share <= 16 else -(-most * share // 32)
    if kh >= 512:
        assert 0 < need <= 8 * len(new) * max(blocks, 2)
    guard = torch.full((need + 4096,), 91, dtype=torch.uint8, device="cuda")
    base._check(rrs, torch, cache, dtype, new, lengths, heads, ws=guard[:need])
    assert (guard[need:] == 91).all()
