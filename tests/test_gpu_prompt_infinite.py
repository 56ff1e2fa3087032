"""GPU tests of Mamba-2 and GDN prompts whose states are not finite: read-outs and states are infinite
or NaN where the recurrence in fp64 has them so, and only there."""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import HALF, _close, _gen, _np, _run_scan, _rrs, _scan_inputs

pytestmark = pytest.mark.gpu


def _same_kind(got, want, tol):
    """Equal infinities, NaN where want has NaN, within tol elsewhere."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(inf, np.isinf(got)) and np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    _close(got[fine], want[fine], np.broadcast_to(tol, want.shape)[fine])


def _check(rrs, torch, kind, lens, t, S0, dims):
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, dims, "bf16")
    with np.errstate(invalid="ignore"):
        want_o, want_S, _ = ref.scan(kind, lens, *map(_np, t), _np(S0))
    # sums of up to 128 products next to states and values of order 1, keys and queries of length 1: 3e-5 of
    # a bound on |S|_F |q|, 1e-5 of one on |S|_F, as for finite ones
    size = np.sqrt(dims[1] * dims[2])
    _same_kind(_np(o), want_o, HALF["bf16"] * np.abs(np.nan_to_num(want_o, posinf=0, neginf=0)) + 3e-5 * size)
    _same_kind(_np(S), want_S, 1e-5 * size)
    return want_o, want_S


def _positive(torch, g, kind, n, heads, dk, dv):
    """Inputs whose keys and queries are positive, so that infinite rows of the state have one sign."""
    q, k, v, beta, gate = _scan_inputs(torch, g, kind, n, heads, 1, dk, dv, "bf16")
    q, k = (torch.nn.functional.normalize(x.float().abs() + 0.01, dim=-1).bfloat16() for x in (q, k))
    return q, k, v, beta, gate


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("small", [False, True])
def test_mamba2_from_infinite_states(dk, dv, small):
    """Infinite elements of a state stay infinite under gates of any size but 0, and reach their column only."""
    rrs, torch = _rrs()
    lens, heads = [70, 40], 2
    g = _gen(torch, dk + dv)
    t = _positive(torch, g, ref.MAMBA2, 110, heads, dk, dv)
    if small:
        t[4][:] = 1e-3  # over a chunk their product underflows
    S0 = torch.randn(2, heads, dk, dv, device="cuda", generator=g)
    S0[0, 0, 5, 7], S0[1, 1, 60, 33], S0[1, 1, 2, 0] = float("inf"), float("-inf"), float("nan")
    o, S = _check(rrs, torch, ref.MAMBA2, lens, t, S0, (heads, dk, dv))
    assert np.isposinf(o[:70, 0, 7]).all() and np.isneginf(S[1, 1, 60, 33]) and np.isfinite(o[:70, 1]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("strong", [False, True])
def test_cut_mamba2_prompts_with_infinite_values(d, strong):
    """An infinite value's column stays infinite through the segments behind it, whatever their gates' product."""
    rrs, torch = _rrs()
    lens, heads = [2600, 1500], 2
    g = _gen(torch, d)
    t = _positive(torch, g, ref.MAMBA2, 4100, heads, d, d)
    if strong:
        t[4][300:] *= 0.5
    t[2][400, 0, 3], t[2][1000, 1, 40], t[2][2600 + 700, 1, 11] = float("inf"), float("-inf"), float("nan")
    S0 = torch.randn(2, heads, d, d, device="cuda", generator=g)
    S0[1, 0, 9, 9] = float("inf")
    o, S = _check(rrs, torch, ref.MAMBA2, lens, t, S0, (heads, d, d))
    assert np.isposinf(o[400:2600, 0, 3]).all() and np.isneginf(S[0, 1, :, 40]).all() and np.isposinf(S[1, 0, 9, 9])


@pytest.mark.parametrize("d", [64, 128])
def test_cut_gdn_prompts_whose_transitions_overflow(d):
    """Keys longer than the delta rule holds, under values of zero: the state is zero until the first
    value, whatever the product of the transitions before it."""
    rrs, torch = _rrs()
    lens, heads = [2600], 2
    g = _gen(torch, 5 * d)
    q, k, v, beta, gate = _scan_inputs(torch, g, ref.GDN, 2600, heads, 1, d, d, "bf16")
    v[:1400] = 0
    k[200:1300] *= 8
    t = (q, k, v, beta, gate)
    o, S = _check(rrs, torch, ref.GDN, lens, t, None, (heads, d, d))
    assert (o[:1400] == 0).all() and np.isfinite(S).all()
    # the states of a second sequence beside it are its own
    more = tuple(torch.cat([x, x[1400:], x[1400:]]) for x in t)
    o, S = _check(rrs, torch, ref.GDN, [2600, 2400], more, None, (heads, d, d))
    assert np.isfinite(S).all()
