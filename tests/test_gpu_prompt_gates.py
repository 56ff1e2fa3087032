"""GPU tests of the gated scan with gates above 1, alone and next to gates of 0, in prompts that run whole
and in prompts long and few enough to be cut into segments.

The scale of the errors is that of the token at hand: a state that large gates blow up and small ones
bring back leaves no error of its large size behind, since an error decays with it. Per token, sums of up to
128 products in fp32 and the gates' roundings, which add up over the tokens like a random walk: 1e-5 of
the largest of |g S|_F before the update and what the update adds, carried along by the gates.
"""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt import HALF, _close, _gen, _np, _run_scan, _rrs, _scan_inputs

pytestmark = pytest.mark.gpu


def _scales(kind, lens, q, k, v, beta, g, S0):
    """Per (token, head) and per (sequence, head): the size of what the read-out and the last state are sums of."""
    heads, dv = v.shape[1:]
    of = np.arange(heads) // (heads // k.shape[1])
    per_token, last, at = np.zeros(v.shape[:2]), np.zeros((len(lens), heads)), 0
    for b, n in enumerate(lens):
        s = np.zeros((heads, k.shape[2], dv)) if S0 is None else S0[b].copy()
        size = np.sqrt((s * s).sum((1, 2)))
        for t in range(at, at + n):
            gt = g[t][:, :, None] if kind == ref.KDA else g[t][:, None, None]
            s, size = s * gt, size * gt.max((1, 2))
            kt = k[t][of]
            w = v[t] - (np.einsum("hi,hij->hj", kt, s) if kind != ref.MAMBA2 else 0)
            add = kt[:, :, None] * (beta[t][:, None] * w)[:, None, :]
            size = np.maximum(size, np.maximum(np.sqrt((s * s).sum((1, 2))), np.sqrt((add * add).sum((1, 2)))))
            s = s + add
            per_token[t] = size * np.sqrt((q[t][of] ** 2).sum(1))
        last[b] = size
        at += n
    return per_token, last


def _check(rrs, torch, kind, lens, t, S0, dims, dtype):
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, dims, dtype)
    n = tuple(map(_np, t))
    want_o, want_S, _ = ref.scan(kind, lens, *n, _np(S0))
    per_token, last = _scales(kind, lens, *n, _np(S0))
    _close(_np(o), want_o, HALF[dtype] * np.abs(want_o) + 3e-5 * per_token[:, :, None])
    err = np.sqrt(((_np(S) - want_S) ** 2).sum((2, 3)))
    assert (err <= 1e-5 * last).all(), f"state off by {np.max(err / last):.3e}"


def _gates_above_one(gate, at):
    """In place, from row `at` on: growth and decay that cancel, a 0 before a large gate and a large one before a 0."""
    gate[at:at + 6] = 1.5
    gate[at + 6:at + 12] = 1 / 1.5
    gate[at + 40], gate[at + 41], gate[at + 50] = 0.0, 2.0 ** 90, 2.0 ** -90
    gate[at + 62], gate[at + 70], gate[at + 71] = 2.0 ** 60, 0.0, 3.0
    gate[at + 80:at + 84] = 2.0 ** -20
    gate[at + 84:at + 88] = 2.0 ** 20


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_gates_above_one(kind, dtype, dk, dv):
    rrs, torch = _rrs()
    lens, heads = [100, 0, 250], 2
    g = _gen(torch, 7 * kind + dk + dv)
    t = _scan_inputs(torch, g, kind, sum(lens), heads, 2, dk, dv, dtype)
    t[4][:, 1:] **= 0.5
    _gates_above_one(t[4], 5)
    _gates_above_one(t[4][:, 1:], 130)
    _gates_above_one(t[4][:, :1], 220)
    # nothing of the state before a 0 comes back, where nothing new covers it
    t[3][318:348] = 0
    t[4][318:348] = 1
    t[4][320], t[4][330], t[4][340] = 0.0, 2.0 ** 100, 2.0 ** 100
    S0 = torch.randn(3, heads, dk, dv, device="cuda", generator=g)
    _check(rrs, torch, kind, lens, t, S0, (heads, dk, dv), dtype)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("d", [64, 128])
def test_gates_above_one_in_cut_prompts(kind, d):
    """The same in the first, an inner and the last segment, and a 0 behind which the gates
    multiply to 2^200: nothing of the state before it comes back."""
    rrs, torch = _rrs()
    lens, heads = [3000], 2
    g = _gen(torch, kind + d)
    t = _scan_inputs(torch, g, kind, 3000, heads, 1, d, d, "bf16")
    for at in (10, 1250, 2850):
        _gates_above_one(t[4], at)
    t[3][1600:1700] = 0
    t[4][1600], t[4][1650], t[4][1660] = 0.0, 2.0 ** 100, 2.0 ** 100
    S0 = torch.randn(1, heads, d, d, device="cuda", generator=g)
    _check(rrs, torch, kind, lens, t, S0, (heads, d, d), "bf16")


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("d", [64, 128])
def test_small_gates_in_cut_prompts(kind, d):
    """Gates of 0, subnormal ones and strong decay in several segments."""
    rrs, torch = _rrs()
    lens, heads = [2700, 1300], 2
    g = _gen(torch, 19 * kind + d)
    t = _scan_inputs(torch, g, kind, 4000, heads, 2, d, d, "bf16")
    gate = t[4]
    gate[100], gate[700:702], gate[1300] = 0.0, 0.0, 1e-42
    gate[1600:1700] = torch.exp(-12.0 * torch.rand(100, heads, device="cuda", generator=g))
    gate[2000:2004] = 1e-30
    gate[3000:3400] = 0.5
    gate[3800], gate[3999] = 0.0, 0.0
    S0 = torch.randn(2, heads, d, d, device="cuda", generator=g)
    _check(rrs, torch, kind, lens, t, S0, (heads, d, d), "bf16")


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_gates_around_one(kind, dk, dv):
    """Growth and decay that nearly cancel, and runs of both whose products stay within 2^50 over 32 tokens and pass it."""
    rrs, torch = _rrs()
    lens, heads = [300, 200], 2
    g = _gen(torch, 11 * kind + dk)
    t = _scan_inputs(torch, g, kind, 500, heads, 1, dk, dv, "bf16")
    gate = t[4]
    gate[:] = 2.0 ** (torch.rand(gate.shape, device="cuda", generator=g) - 0.5)
    gate[64:94], gate[96:126] = 2.0, 0.5
    gate[300:348], gate[350:398] = 3.0, 1 / 3.0  # 2^50.7 in a chunk and more
    S0 = torch.randn(2, heads, dk, dv, device="cuda", generator=g)
    _check(rrs, torch, kind, lens, t, S0, (heads, dk, dv), "bf16")
