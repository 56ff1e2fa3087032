"""GPU tests of how exactly the chunked scan keeps the states of bf16 GDN and Mamba-2 prompts.

The bound on the relative error of a head's state, in the Frobenius norm. Every token rounds each
element of the state a fixed number of times m: its gate's power (2 half-steps of 2^-24), the product with it,
the sums of W (4: its right-hand side, the products with T) and the addition to the state (2): m = 9. With gates
of 0.9 to 1, 0.95 on average, a rounding lives for 1 / (1 - 0.95^2) = 10 tokens in the sum of squares, and
roundings are independent: sqrt(9 x 10) half-steps, each of rms 2^-24 / sqrt(3), is 3.3e-7. The bound is
5e-7. An operand cut to 16 bits instead is off by up to 2^-18, rms 2^-18 / sqrt(3), in every
token: 64 half-steps, sqrt(10) of them over the state's memory, 7e-6. The emulation in
test_prompt_pieces.py shows both on the CPU.
"""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import _check_scan, _gen, _np, _run_scan, _rrs, _scan_inputs

pytestmark = pytest.mark.gpu

BOUND = 5e-7


def _check(rrs, torch, kind, lens, heads, kh, dk, dv, seed):
    g = _gen(torch, seed)
    t = _scan_inputs(torch, g, kind, sum(lens), heads, kh, dk, dv, "bf16")
    S0 = torch.randn(len(lens), heads, dk, dv, device="cuda", generator=g)
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, (heads, dk, dv), "bf16")
    want = ref.scan(kind, lens, *map(_np, t), _np(S0))
    _check_scan(_np(o), _np(S), want, "bf16")
    err = np.sqrt(((_np(S) - want[1]) ** 2).sum((2, 3)))
    top = np.sqrt((want[1] ** 2).sum((2, 3)))
    assert (err <= BOUND * top).all(), f"{np.max(err / top):.2e}"
    for b, n in enumerate(lens):
        if n == 0:
            assert np.array_equal(_np(S)[b], _np(S0)[b])


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_whole_prompts(kind, dk, dv):
    rrs, torch = _rrs()
    _check(rrs, torch, kind, [700, 32, 257, 64], 2, 1, dk, dv, dk + dv)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("d", [64, 128])
def test_cut_prompts(kind, d):
    rrs, torch = _rrs()
    _check(rrs, torch, kind, [2600, 1400], 2, 2, d, d, d)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64)])
def test_more_sequences_than_are_ranked(kind, dk, dv):
    """140 prompts of 0 to 63 tokens, which run in the order given."""
    rrs, torch = _rrs()
    lens = np.random.default_rng(dv).integers(0, 64, 140)
    lens[[0, 70, 139]] = 0
    assert lens.sum() >= 16 * 140
    _check(rrs, torch, kind, lens.tolist(), 2, 1, dk, dv, 3 * dk + dv)
