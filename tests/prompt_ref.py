"""Plain fp64 forms of the prompt path (short convolution, gated scan, row norm), written from the
definitions and used by the tests only. Arrays are numpy float64."""
from __future__ import annotations

import numpy as np

GDN, KDA, MAMBA2 = 0, 1, 2


def silu(z):
    return z / (1.0 + np.exp(-z))


def conv(x, lens, weight, bias, window, act):
    """x [tokens, channels]; window [batch, width - 1, channels] or None. Returns y, the new windows
    and, per output, the sum of the absolute terms (the scale of its rounding errors)."""
    width, ch = weight.shape
    y, mag = np.zeros_like(x), np.zeros_like(x)
    out = np.zeros((len(lens), width - 1, ch))
    at = 0
    for b, n in enumerate(lens):
        past = window[b] if window is not None else np.zeros((width - 1, ch))
        line = np.concatenate([past, x[at:at + n]])
        for t in range(n):
            terms = weight * line[t:t + width]
            b0 = bias if bias is not None else np.zeros(ch)
            s = b0 + terms.sum(0)
            y[at + t] = silu(s) if act else s
            mag[at + t] = np.abs(b0) + np.abs(terms).sum(0)
        out[b] = line[n:]
        at += n
    return y, out, mag


def scan(kind, lens, q, k, v, beta, g, S0):
    """q, k [tokens, key_heads, d_k]; v [tokens, heads, d_v]; beta [tokens, heads]; g [tokens, heads]
    (KDA: [tokens, heads, d_k]); S0 [batch, heads, d_k, d_v] or None. Returns o, the final states
    and, per (token, head), |q_t| times the largest |S|_F (and |beta v| row, whose sum it is) so far:
    the scale of a read-out's errors."""
    heads, dv = v.shape[1], v.shape[2]
    kh, dk = k.shape[1], k.shape[2]
    of = np.arange(heads) // (heads // kh)
    o = np.zeros_like(v)
    mag = np.zeros(v.shape[:2])
    S = np.zeros((len(lens), heads, dk, dv))
    at = 0
    for b, n in enumerate(lens):
        s = np.zeros((heads, dk, dv)) if S0 is None else S0[b].copy()
        top = np.sqrt((s * s).sum((1, 2)))
        for t in range(at, at + n):
            s = s * (g[t][:, :, None] if kind == KDA else g[t][:, None, None])
            kt, qt = k[t][of], q[t][of]
            w = v[t]
            if kind != MAMBA2:
                w = w - np.einsum("hi,hij->hj", kt, s)
            s = s + kt[:, :, None] * (beta[t][:, None] * w)[:, None, :]
            o[t] = np.einsum("hi,hij->hj", qt, s)
            top = np.maximum(top, np.sqrt((s * s).sum((1, 2))))
            mag[t] = top * np.sqrt((qt * qt).sum(1))
        S[b] = s
        at += n
    return o, S, mag


def norm_rows(x, weight, gate, eps, gate_first, skip, scale):
    """x [rows, heads, dim]. Returns y, x + scale skip and the scale of y's rounding errors."""
    t, mag = x, np.abs(x)
    if skip is not None:
        sc = np.ones(x.shape[1]) if scale is None else scale
        t = x + sc[None, :, None] * skip
        mag = mag + np.abs(sc[None, :, None] * skip)
    z = silu(gate) if gate is not None else 1.0
    u = t * z if gate is not None and gate_first else t
    inv = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return t * z * inv * weight, t, mag * np.abs(z) * inv * np.abs(weight)
