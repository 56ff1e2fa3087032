"""GPU tests of how exactly bf16 GDN and Mamba-2 prompts are computed: every product with a state or a
value takes fp32 operands, in the chunked scan too.

Read-outs that cancel show the operands' bits, which rounding the result to bf16 hides otherwise: a
read-out of size 2^-13 is rounded to bf16 at 2^-22, and what is left of an error of its terms (of
size 1) shows above that. Fp32 arithmetic puts a few half-steps of 2^-24 into each term: a gate's
logarithm and power (4), two products (2), the last piece of an operand cut to 24 bits (1), the sum's own
roundings (4). 2^-20 of the absolute terms is 16 of them. An operand cut to 16 bits is off by up to
2^-18 of a term, 64 of them.
"""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import HALF, _close, _gen, _np, _run_scan, _rrs

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_readouts_that_cancel_over_the_state(kind, dk, dv):
    """q reads two rows of a state that is carried along unchanged, the second the first's negative up to 2^-13."""
    rrs, torch = _rrs()
    lens, heads = [40, 70], 3
    n = sum(lens)
    g = _gen(torch, dk + 2 * dv)
    S0 = torch.randn(2, heads, dk, dv, device="cuda", generator=g)
    S0[:, :, 1::2] = S0[:, :, 0::2] * (2.0 ** -13 * torch.randn(2, heads, dk // 2, dv, device="cuda", generator=g) - 1)
    pair = torch.randint(0, dk // 2, (n,), device="cuda", generator=g)
    q = torch.zeros(n, 1, dk, device="cuda")
    q[torch.arange(n), 0, 2 * pair] = 1
    q[torch.arange(n), 0, 2 * pair + 1] = 1
    k = torch.nn.functional.normalize(torch.randn(n, 1, dk, device="cuda", generator=g), dim=-1)
    v = torch.randn(n, heads, dv, device="cuda", generator=g)
    t = (q.bfloat16(), k.bfloat16(), v.bfloat16(), torch.zeros(n, heads, device="cuda"), torch.ones(n, heads, device="cuda"))
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, (heads, dk, dv), "bf16")
    assert torch.equal(S, S0)
    want, _, _ = ref.scan(kind, lens, *map(_np, t), _np(S0))
    own = _np(S0)[np.repeat([0, 1], lens)]  # the states that the tokens read
    terms = np.einsum("ti,thij->thj", _np(q)[:, 0], np.abs(own))
    _close(_np(o), want, HALF["bf16"] * np.abs(want) + 2.0 ** -20 * terms)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_readouts_that_cancel_over_two_tokens(kind, dk, dv):
    """Two tokens of one key, whose values cancel up to 2^-13 in the second one's read-out; every pair
    of tokens has a key channel of its own."""
    rrs, torch = _rrs()
    heads, n = 4, 2 * dk
    g = _gen(torch, 3 * dk + dv)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, device="cuda", generator=g)

    k = torch.zeros(n, 1, dk, device="cuda")
    k[torch.arange(n), 0, torch.arange(n) // 2] = 1
    v = torch.randn(n, heads, dv, device="cuda", generator=g).bfloat16()
    v[1::2] = -v[0::2]
    beta, gate = uniform(0.3, 0.9, n, heads), torch.ones(n, heads, device="cuda")
    gate[1::2] = uniform(0.6, 1.0, dk, heads)
    first = gate[1::2] * beta[0::2]
    even = first if kind == ref.MAMBA2 else first / (1 + first)
    beta[1::2] = even * (1 + 2.0 ** -13 * torch.randn(dk, heads, device="cuda", generator=g))
    t = (k.bfloat16(), k.bfloat16(), v, beta, gate)
    o, _ = _run_scan(rrs, torch, kind, [n], t, None, (heads, dk, dv), "bf16")
    want, _, _ = ref.scan(kind, [n], *map(_np, t), None)
    tol = HALF["bf16"] * np.abs(want)
    # the value of the first token, and of the second with what the delta rule takes from it
    tol[0::2] += 2.0 ** -20 * np.abs(want[0::2])
    size = np.abs(_np(v)[0::2])
    f, b = _np(first)[:, :, None], _np(beta)[1::2][:, :, None]
    tol[1::2] += 2.0 ** -20 * size * (f + b if kind == ref.MAMBA2 else f + b + b * f)
    _close(_np(o), want, tol)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_keys_that_cancel_over_the_state(dk, dv):
    """The delta rule's own read: every key reads two rows of the state, one the other's negative up to
    2^-13, and puts what it read back. Sums of three pieces for each of two rows and three additions to the
    state, 10 half-steps of 2^-24 of a row's value: 2^-20 is 16; a row cut to 16 bits is off by up to 64."""
    rrs, torch = _rrs()
    heads, n = 3, dk // 2
    g = _gen(torch, 5 * dk + dv)
    S0 = torch.randn(1, heads, dk, dv, device="cuda", generator=g)
    S0[:, :, 1::2] = S0[:, :, 0::2] * (2.0 ** -13 * torch.randn(1, heads, n, dv, device="cuda", generator=g) - 1)
    k = torch.zeros(n, 1, dk, device="cuda")
    k[torch.arange(n), 0, 2 * torch.arange(n)] = 1
    k[torch.arange(n), 0, 2 * torch.arange(n) + 1] = 1
    v = torch.zeros(n, heads, dv, device="cuda")
    ones = torch.ones(n, heads, device="cuda")
    t = (k.bfloat16(), k.bfloat16(), v.bfloat16(), ones, ones)
    _, S = _run_scan(rrs, torch, ref.GDN, [n], t, S0, (heads, dk, dv), "bf16")
    _, want, _ = ref.scan(ref.GDN, [n], *map(_np, t), _np(S0))
    _close(_np(S), want, 2.0 ** -20 * np.abs(_np(S0)))
