"""GPU tests of a layer's prompt with the convolution's output as keys and queries, brought to unit length
in place by seed_norm_rows as the delta rule needs it, with beta up to 1."""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import HALF, _check_scan, _close, _gen, _np, _offsets, _rrs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
def test_delta_rule_behind_the_convolution(kind, dk, dv):
    rrs, torch = _rrs()
    g = _gen(torch, 7 * dk + kind)
    lens, heads, key_heads = [400, 0, 1, 130], 4, 2
    n, hk = sum(lens), key_heads * dk
    channels = 2 * hk + heads * dv
    off = _offsets(torch, lens)
    x = torch.randn(n, channels, device="cuda", generator=g).bfloat16()
    weight = torch.randn(4, channels, device="cuda", generator=g)
    y, window = torch.empty_like(x), torch.empty(len(lens), 3, channels, dtype=x.dtype, device="cuda")
    rrs.seed_prefill_conv(rrs.make_conv(len(lens), channels, 4), x, off, weight, None, window, y)
    q, k = (y[:, i * hk:(i + 1) * hk].view(n, key_heads, dk) for i in range(2))
    v = y[:, 2 * hk:].view(n, heads, dv)
    before = [_np(t) for t in (q, k)]
    values = v.clone()
    unit = torch.full((key_heads, dk), dk ** -0.5, device="cuda")
    for t, old in zip((q, k), before):
        rrs.seed_norm_rows(t, unit, t)
        want, _, mag = ref.norm_rows(old, _np(unit), None, 1e-6, False, None, None)
        _close(_np(t), want, HALF["bf16"] * np.abs(want) + 2.0 ** -18 * mag)
        # every value is off by at most half a bf16 step, and eps takes d_k eps / |x|^2 away
        length = np.linalg.norm(_np(t), axis=-1)
        assert (np.abs(length - 1) <= 2.0 ** -7 + dk * 1e-6 / (old * old).sum(-1)).all()
    assert torch.equal(v, values)
    beta = torch.rand(n, heads, device="cuda", generator=g)
    gate = 1 - 0.1 * torch.rand(*((n, heads, dk) if kind == ref.KDA else (n, heads)), device="cuda", generator=g)
    shape = rrs.make_shape(kind, len(lens), heads, dk, dv, 8, 8, rrs.SEED_BF16)
    S = torch.empty(len(lens), heads, dk, dv, device="cuda")
    o = torch.empty(n, heads, dv, dtype=torch.bfloat16, device="cuda")
    rrs.seed_prefill_scan(shape, off, q, k, v, beta, gate, S, o)
    want = ref.scan(kind, lens, *map(_np, (q, k, v, beta, gate)), None)
    _check_scan(_np(o), _np(S), want, "bf16")
    # |S| never grows by more than beta |k| |v| a token, under gates of at most 1
    assert np.linalg.norm(_np(S), axis=(2, 3)).max() <= 1.02 * sum(np.linalg.norm(_np(v), axis=-1).max(-1))
