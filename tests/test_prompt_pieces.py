"""The precision of the chunked scan's arithmetic, emulated on the CPU: fp32 operands as sums of three bf16
pieces keep the states of GDN and Mamba-2 prompts within the bound that test_gpu_prompt_states.py
holds the kernels to, and two pieces of T and its right-hand side, or of W, do not. (Two of the state where
it meets k stay within it on random data, where the sum over the key evens them out:
test_gpu_prompt_precision.py has states that cancel there.)"""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref
from test_gpu_prompt_states import BOUND

C, F = 32, np.float32


def _bf16(x):
    u = np.ascontiguousarray(x, F).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)).view(F)


def _pieces(x, n):
    out, rest = [], x.astype(F)
    for _ in range(n):
        out.append(_bf16(rest))
        rest = rest - out[-1]
    return out


def _product(a, b):
    """a b with a's and b's pieces: the products whose order is below 3, smallest first, summed in fp32."""
    acc = np.zeros((a[0].shape[0], b[0].shape[1]), F)
    for order in (2, 1, 0):
        for i, x in enumerate(a):
            for j, y in enumerate(b):
                if i + j == order:
                    acc = acc + x @ y
    return acc


def _chunks(kind, k, v, beta, g, S, n_state, n_solve, n_update):
    """The state after the chunked recurrence: pieces of the state where it meets k, of T and its
    right-hand side, and of W where it enters the state."""
    for t in range(0, len(k), C):
        kc, vc, b = k[t:t + C].astype(F), v[t:t + C].astype(F), beta[t:t + C].astype(F)[:, None]
        c = np.cumsum(np.log2(g[t:t + C]))
        head, tail = (2.0 ** c).astype(F)[:, None], (2.0 ** (c[-1] - c)).astype(F)[:, None]
        if kind == ref.GDN:
            L = np.tril((b * (2.0 ** (c[:, None] - c[None])).astype(F)) * (kc @ kc.T), -1)
            T = np.linalg.inv(np.eye(C) + L.astype(float)).astype(F) * b.T
            rhs = vc - head * _product([kc], _pieces(S, n_state))
            w = _product(_pieces(T, n_solve), _pieces(rhs, n_solve))
        else:
            w = b * vc
        S = head[-1] * S + _product([kc.T], _pieces(tail * w, n_update))
    return S


def _error(kind, *pieces):
    r = np.random.default_rng(5)
    n, dk, dv = 704, 128, 128
    k, v = r.standard_normal((n, dk)), r.standard_normal((n, dv))
    if kind == ref.GDN:
        k /= np.linalg.norm(k, axis=1, keepdims=True)
    k, v = _bf16(k).astype(float), _bf16(v).astype(float)
    beta, g = r.random(n).astype(F).astype(float), (1 - 0.1 * r.random(n)).astype(F).astype(float)
    S0 = r.standard_normal((dk, dv)).astype(F)
    _, want, _ = ref.scan(kind, [n], k[:, None], k[:, None], v[:, None], beta[:, None], g[:, None], S0[None, None].astype(float))
    got = _chunks(kind, k, v, beta, g, S0, *pieces)
    return np.linalg.norm(got - want[0, 0]) / np.linalg.norm(want)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
def test_three_pieces_hold_the_bound(kind):
    assert _error(kind, 3, 3, 3) <= BOUND


@pytest.mark.parametrize("kind,pieces", [(ref.GDN, (3, 2, 3)), (ref.GDN, (3, 3, 2)), (ref.GDN, (2, 2, 2)), (ref.MAMBA2, (3, 3, 2))])
def test_two_pieces_break_it(kind, pieces):
    assert _error(kind, *pieces) > BOUND
