"""Plain fp64 forms of the attention layers' operators and of draft verification, written from the
definitions and used by the tests only. Arrays are numpy float64."""
from __future__ import annotations

import math

import numpy as np


def turns(dim, base=10000.0, kind="plain", factor=1.0, length=0.0, low=1.0, high=32.0):
    out = []
    if kind == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    for i in range(dim // 2):
        f = 1.0 / base ** (2 * i / dim)  # radians per position
        if kind == "linear":
            f /= factor
        elif kind == "parts":
            n = length * f / (2 * math.pi)
            keep = min(max((n - low) / (high - low), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        elif kind == "index":
            def at(n):  # the index whose pair makes n turns over the trained length
                return dim * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(math.floor(at(high)), 0), min(math.ceil(at(low)), dim - 1)
            keep = 1 - min(max((i - a) / (b - a), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        out.append(f / (2 * math.pi))
    return np.array(out)


def rotate(x, positions, t, interleaved=False, amplitude=1.0):
    """x [rows, heads, dim]. Returns y and, per value, the sum of its absolute terms."""
    y, mag, rot = x.copy(), np.zeros_like(x), 2 * len(t)
    angle = 2 * math.pi * np.mod(positions[:, None].astype(np.float64) * t, 1.0)
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    mag[..., one] = mag[..., two] = abs(amplitude) * (np.abs(a) + np.abs(b))
    return y, mag


def attend(q, K, V, positions, scale, window=0, there=None):
    """One request and key head: q [rows, dim] at positions [rows], K, V [keys, dim]; there: bool [keys],
    positions that are there. Returns o, lse, the weighted mean of |v| and the largest sum of |q k| scale."""
    rows, dim = q.shape
    o, lse = np.zeros((rows, dim)), np.full(rows, -np.inf)
    mag, top = np.zeros((rows, dim)), np.zeros(rows)
    for r in range(rows):
        j = np.arange(len(K))
        seen = (j <= positions[r]) & ((j > positions[r] - window) if window else True)
        if there is not None:
            seen &= there
        if not seen.any():
            continue
        s = scale * (K[seen] @ q[r])
        m = s.max()
        if m == -np.inf:
            continue
        w = np.exp(s - m)
        o[r] = (w @ V[seen]) / w.sum()
        lse[r] = m + math.log(w.sum())
        mag[r] = (w @ np.abs(V[seen])) / w.sum()
        top[r] = abs(scale) * (np.abs(K[seen]) @ np.abs(q[r])).max()
    return o, lse, mag, top


def verify(target, draft, drafts, uniforms, draws, offsets):
    """Returns out (-2: a row that is not written) and counts."""
    out, counts = np.full(len(target), -2), []
    vocab = target.shape[1]
    for b in range(len(offsets) - 1):
        lo, hi = offsets[b], offsets[b + 1]
        if hi <= lo:
            counts.append(0)
            continue
        r = lo
        while r < hi - 1:
            x = drafts[r]
            if not 0 <= x < vocab:
                break
            if not uniforms[r] * (draft[r, x] if draft is not None else 1.0) < target[r, x]:
                break
            out[r] = x
            r += 1
        w = target[r].copy()
        if r < hi - 1 and draft is not None:
            w = w - draft[r]
        elif r < hi - 1 and 0 <= drafts[r] < vocab:
            w[drafts[r]] = 0
        for w in (w, target[r]):
            w = np.where(w > 0, w, 0.0)
            if w.sum() > 0:
                break
        token = -1
        if w.sum() > 0:
            cum = np.cumsum(w)
            hit = np.nonzero((cum > draws[b] * cum[-1]) & (w > 0))[0]
            token = hit[0] if len(hit) else np.nonzero(w > 0)[0][-1]
        out[r] = token
        out[r + 1:hi] = -1
        counts.append(r - lo + 1)
    return out, np.array(counts)
