"""GPU tests of the attention layers (seed_rotate_rows, seed_cache_append, seed_decode_attend) against
the plain fp64 forms of attend_ref.py, which receive exactly the values the device buffers hold.

Tolerances, element by element. A value rounded once to its format is off by at most half a step,
eps / 2 of its size (bf16 2^-8, fp32 2^-24). Before that rounding:
  - rotation: the reduced angle (at most half a turn) rounds to fp32, 2^-24 pi; sine and cosine are good to
    2^-22, two products and a sum follow: 2^-20 of the sum of the absolute terms;
  - attention: a score is a sum of dim products in fp32, off by at most dim 2^-24 of the sum of its absolute terms A
    (the scale's rounding and the exponential's argument are within it), so a weight by that much of itself and o
    by twice that of the weighted mean M of |v|; weights in two bf16 pieces, 2^-16 M; a sum over n keys in runs of
    128 and 32 at a time, (n / 4 + 64) 2^-24 M. lse by dim 2^-24 A, and its own rounding and logarithm, 2^-22 of 1 + |lse|.
"""
from __future__ import annotations

import numpy as np
import pytest

import attend_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _rrs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_recurrent_state_amd as rrs
    return rrs, torch


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(torch, values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _offsets(torch, lens, start=0):
    return _i32(torch, np.concatenate([[start], start + np.cumsum(lens)]))


def _close(got, want, tol):
    bad = ~((np.abs(got - want) <= tol) | (got == want))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off; worst {np.abs(got - want)[bad].max():.3e} at {np.argwhere(bad)[0]}"


# ---- rotation -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (5, 3, 72, 20), (67, 5, 80, 80), (33, 8, 128, 64),
                                                (700, 40, 128, 128), (9, 4, 256, 64), (129, 1, 64, 48), (3, 7, 100, 30)])
def test_rotate_rows(dtype, interleaved, rows, heads, dim, rot):
    rrs, torch = _rrs()
    g = _gen(torch, rows + dim + rot)
    dt = _dt(torch, dtype)
    rotary = rrs.make_rotary(rot, base=500000.0, interleaved=interleaved, amplitude=1.25)
    t = ref.turns(rot, base=500000.0)
    far = torch.randint(-1000, 1 << 21, (rows,), generator=g, device="cuda", dtype=torch.int32)
    far[0] = (1 << 31) - 1
    far[-1] = -(1 << 31) if rows > 1 else 0
    wide = torch.randn(rows, heads * dim + 24, generator=g, device="cuda").to(dt)
    x = wide[:, 8:8 + heads * dim].view(rows, heads, dim) if dim > 2 else wide[:, :2].view(rows, 1, 2)
    want, mag = ref.rotate(_np(x), far.cpu().numpy(), t, interleaved, 1.25)
    tol = HALF[dtype] * np.abs(want) + 2.0 ** -20 * mag
    before = wide.clone()
    y = torch.full((rows + 2, heads, dim), 7.0, dtype=dt, device="cuda")
    rrs.seed_rotate_rows(rotary, x, far, y[1:-1])
    _close(_np(y[1:-1]), want, tol)
    assert (y[0] == 7.0).all() and (y[-1] == 7.0).all() and torch.equal(wide, before)
    rrs.seed_rotate_rows(rotary, x, far, x)  # in place: the columns around stay
    assert torch.equal(x, y[1:-1].contiguous().view_as(x))
    wide.view(-1)[0] = before.view(-1)[0]
    assert torch.equal(wide[:, 8 + heads * dim:], before[:, 8 + heads * dim:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rot", [(5, 40, 128, 100), (2100, 40, 128, 98), (3, 64, 72, 72), (2050, 64, 72, 36), (7, 80, 256, 158),
                                                (2049, 72, 256, 64), (2, 3, 2048, 14), (2, 2, 1032, 1030), (1, 1, 16, 2)])
def test_rotate_parts_of_any_size(dtype, interleaved, rows, heads, dim, rot):
    """Turned parts that do not divide into 16 bytes, over several turns of a workgroup and many values a token; what lies
    behind them keeps its bits, in place too."""
    test_rotate_rows(dtype, interleaved, rows, heads, dim, rot)
    rrs, torch = _rrs()
    rotary = rrs.make_rotary(rot, interleaved=interleaved)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    x = torch.randint(-(1 << 15), 1 << 15, (3, heads, dim), generator=_gen(torch, 1), device="cuda", dtype=torch.int32).to(bits)
    x[..., :rot] = 0
    x[..., rot:] |= 0x7f81 if dtype == "bf16" else 0x7f800001  # NaN of all kinds
    before, y = x.clone(), torch.zeros_like(x)
    at = _i32(torch, [0, 5, -9])
    rrs.seed_rotate_rows(rotary, x.view(_dt(torch, dtype)), at, y.view(_dt(torch, dtype)))
    zero = y.view(_dt(torch, dtype))[..., :rot] == 0  # of either sign: 0 c - 0 s
    assert torch.equal(y[..., rot:], before[..., rot:]) and zero.all()
    rrs.seed_rotate_rows(rotary, x.view(_dt(torch, dtype)), at, x.view(_dt(torch, dtype)))
    assert torch.equal(x[..., rot:], before[..., rot:])


def test_rotation_keeps_products():
    """Turned queries and keys meet as the difference of their positions says, also far out."""
    rrs, torch = _rrs()
    rotary = rrs.make_rotary(128, interleaved=True)
    g = _gen(torch, 3)
    x = torch.randn(2, 1, 128, generator=g, device="cuda")
    dots = []
    for shift in (0, 1000, 1 << 20, 1 << 30):
        y = torch.empty_like(x)
        rrs.seed_rotate_rows(rotary, x, _i32(torch, [5 + shift, 77 + shift]), y)
        dots.append(float(_np(y[0, 0]) @ _np(y[1, 0])))
    mass = float(np.abs(_np(x[0, 0])) @ np.abs(_np(x[1, 0])))
    assert max(dots) - min(dots) <= 2.0 ** -18 * mass * 2, dots


# ---- the cache ------------------------------------------------------------------------------------

def _cache(rrs, torch, lengths, kh, dim, page, dtype, seed, layout="tokens", fill=None, spare=3):
    """A pool with pages in random order, filled with random values (or `fill`)."""
    g = _gen(torch, seed)
    dt = _dt(torch, dtype)
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n

    def make():
        shape = {"tokens": (pool, page, kh, dim), "heads": (pool, kh, page, dim)}.get(layout)
        if shape is None:
            return None
        x = torch.randn(shape, generator=g, device="cuda").to(dt)
        if fill is not None:
            x.fill_(fill)
        return x if layout == "tokens" else x.transpose(1, 2)

    if layout == "both":  # keys and values of a page in one buffer
        x = torch.randn(pool, page, 2, kh, dim, generator=g, device="cuda").to(dt)
        if fill is not None:
            x.fill_(fill)
        k, v = x[:, :, 0], x[:, :, 1]
    else:
        k, v = make(), make()
    return rrs.Cache(k, v, table)


def _gather(cache, b, n):
    """Request b's first n keys and values [n, heads, dim]; pages that are not there read as page 0."""
    import torch
    j = torch.arange(n, device="cuda")
    page = cache.k.shape[1]
    number = cache.table[b].long()[j // page]
    number = torch.where((number >= 0) & (number < cache.k.shape[0]), number, 0)
    return cache.k[number, j % page], cache.v[number, j % page]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("new,history,heads,kh,dim,page,rot,interleaved", [
    ([1], [0], 4, 4, 64, 16, 64, False),
    ([1] * 70, None, 8, 2, 128, 32, 128, False),
    ([0, 3, 0, 0, 17, 1, 0], [5, 13, 0, 2, 15, 1, 1], 6, 2, 128, 16, 32, True),
    ([40, 700, 3], [0, 9, 100], 16, 2, 256, 64, 64, False),
    ([2, 2], [31, 1], 3, 3, 64, 16, 6, True),
    ([1, 0, 5], [4, 4, 4], 2, 1, 128, 16, None, False),
])
def test_cache_append(dtype, layout, new, history, heads, kh, dim, page, rot, interleaved):
    rrs, torch = _rrs()
    g = _gen(torch, len(new) + dim)
    dt = _dt(torch, dtype)
    history = list(range(len(new))) if history is None else history
    lengths = [a + b for a, b in zip(new, history)]
    cache = _cache(rrs, torch, lengths, kh, dim, page, dtype, 11, layout)
    lead, n = 2, sum(new)
    total = lead + n + 3
    odd = 3 if rot == 6 else 0  # rows that allow no 16-byte access
    buf = torch.randn(total, (heads + 2 * kh) * dim + odd, generator=g, device="cuda").to(dt)
    q, k, v = (buf[:, a * dim:b * dim].view(total, b - a, dim) for a, b in ((0, heads), (heads, heads + kh), (heads + kh, heads + 2 * kh)))
    rotary = rrs.make_rotary(rot, interleaved=interleaved) if rot else None
    t = ref.turns(rot) if rot else np.zeros(0)
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(new, lengths)] + [np.zeros(0)]).astype(np.int64)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    kr, kmag = ref.rotate(_np(k[lead:lead + n]), pos, t, interleaved)
    qr, qmag = ref.rotate(_np(q[lead:lead + n]), pos, t, interleaved)
    out = torch.full((total, heads, dim), 7.0, dtype=dt, device="cuda")
    rrs.seed_cache_append(cache, _i32(torch, lengths), k, v, offsets=_offsets(torch, new, lead), rotary=rotary, q=q, q_out=out)
    assert (out[:lead] == 7.0).all() and (out[lead + n:] == 7.0).all()
    _close(_np(out[lead:lead + n]), qr, HALF[dtype] * np.abs(qr) + 2.0 ** -20 * qmag)
    at, seq = 0, []
    for b, m in enumerate(new):
        got, gv = _gather(cache, b, lengths[b])
        _close(_np(got[history[b]:]), kr[at:at + m], HALF[dtype] * np.abs(kr[at:at + m]) + 2.0 ** -20 * kmag[at:at + m])
        assert torch.equal(gv[history[b]:], v[lead + at:lead + at + m])
        j = torch.arange(history[b], lengths[b], device="cuda")  # everything else in the pool is as it was
        number = cache.table[b].long()[j // page]
        want_k[number, j % page], want_v[number, j % page] = got[history[b]:], gv[history[b]:]
        at += m
    assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
    if n == len(new) and all(m == 1 for m in new):  # the same without offsets, q in place
        again, k1, v1 = q[lead:lead + n].clone(), cache.k.clone(), cache.v.clone()
        rrs.seed_cache_append(cache, _i32(torch, lengths), k[lead:lead + n], v[lead:lead + n], rotary=rotary, q=again, q_out=again)
        assert torch.equal(again, out[lead:lead + n]) and torch.equal(cache.k, k1) and torch.equal(cache.v, v1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,heads,kh,dim,rot", [([3, 0, 40], 64, 8, 256, 64), ([1, 2, 1], 40, 5, 128, 100), ([2, 2200], 12, 1, 64, 58), ([4], 7, 7, 256, 250)])
def test_append_parts_of_any_size(dtype, interleaved, new, heads, kh, dim, rot):
    """Many values a token, and turned parts that do not divide into 16 bytes."""
    test_cache_append(dtype, "heads", new, [5] * len(new), heads, kh, dim, 16, rot, interleaved)


def test_append_places_that_are_not_there():
    """Rows at negative positions, behind the table or in missing pages are not stored; wrong offsets stay inside."""
    rrs, torch = _rrs()
    g = _gen(torch, 9)
    for bad in ([-1, 10 ** 6, 5], [2, 0, -7], [0, -(1 << 31), (1 << 31) - 1]):
        cache = _cache(rrs, torch, [40, 40, 40], 2, 64, 16, "bf16", 4, fill=3.0)
        cache.table[2, 0] = 10 ** 6  # no such page
        cache.table[0, 0] = -5
        k = torch.randn(12, 2, 64, generator=g, device="cuda").bfloat16()
        rrs.seed_cache_append(cache, _i32(torch, bad), k, k.clone(), offsets=_i32(torch, [0, 4, 8, 12]), rotary=rrs.make_rotary(64),
                              q=k, q_out=torch.empty_like(k))
        changed = int((cache.v != 3.0).any(-1).any(-1).sum())
        assert changed == 0, (bad, changed)
    cache = _cache(rrs, torch, [40, 40, 40], 2, 64, 16, "bf16", 4, fill=3.0)
    for offsets in ([5, 3, 9, 100], [-4, 2, 2, 7], [12, 12, 0, 0], [1 << 30, -(1 << 31), 6, 2]):
        out = torch.full_like(k, 7.0)
        rrs.seed_cache_append(cache, _i32(torch, [20, 20, 20]), k, k.clone(), offsets=_i32(torch, offsets), q=k, q_out=out)
        torch.cuda.synchronize()
        assert ((out == 7.0) | (out == k)).all()


# ---- attention ------------------------------------------------------------------------------------

def _check(rrs, torch, cache, dtype, new, lengths, heads, lead=0, scale=None, window=0, max_length=None, most=None, ragged=True,
           seed=1, q=None, ws=None, stream=None):
    """Runs the attention and compares every row with the definition. Returns o and lse."""
    dt, dim, kh = _dt(torch, dtype), cache.k.shape[3], cache.k.shape[2]
    n = sum(new)
    total = lead + n + (2 if ragged else 0)
    if q is None:
        q = torch.randn(total, heads, dim, generator=_gen(torch, seed), device="cuda").to(dt)
    o = torch.full((total, heads, dim), 7.0, dtype=dt, device="cuda")
    lse = torch.full((total, heads), 9.0, device="cuda")
    most = max(max(new), 1) if most is None else most
    rrs.seed_decode_attend(cache, _i32(torch, lengths), q, o, offsets=_offsets(torch, new, lead) if ragged else None, max_tokens=most,
                           max_length=max_length, scale=scale, window=window, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert (o[:lead] == 7.0).all() and (o[lead + n:] == 7.0).all() and (lse[lead + n:] == 9.0).all()
    sc = dim ** -0.5 if scale is None else float(np.float32(scale))
    sc = float(np.float32(sc))
    qn, on, ln = _np(q), _np(o), _np(lse)
    at = lead
    for b, (m, length) in enumerate(zip(new, lengths)):
        if max_length is not None:
            length = min(length, max_length)
        length = max(length, 0)
        K, V = _gather(cache, b, min(length, cache.table.shape[1] * cache.k.shape[1]))
        entries = cache.table[b].cpu().numpy()
        there = np.repeat((entries >= 0) & (entries < cache.k.shape[0]), cache.k.shape[1])[:length]
        K, V = _np(K), _np(V)
        pos = np.arange(length - m, length)
        done = min(m, most)
        for h in range(kh):
            group = slice(h * heads // kh, (h + 1) * heads // kh)
            rows = qn[at:at + done, group].reshape(-1, dim)
            p = np.repeat(pos[:done], heads // kh)
            want, wl, mag, top = ref.attend(rows, K[:, h], V[:, h], p, sc, window, there)
            got, gl = on[at:at + done, group].reshape(-1, dim), ln[at:at + done, group].reshape(-1)
            e = dim * 2.0 ** -24 * top
            with np.errstate(invalid="ignore"):
                tol = HALF[dtype] * np.abs(want) + mag * (2 * e[:, None] + 2.0 ** -16 * (dtype == "bf16") + (length / 4 + 64) * 2.0 ** -24)
                _close(got, want, tol)
                _close(gl, wl, e + 2.0 ** -22 * (1 + np.abs(wl)))
        assert (o[at + done:at + m] == 7.0).all()
        at += m
    return o, lse


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 130, 257, 640, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kh", [(1, 1), (12, 4), (16, 1), (40, 2)])
def test_one_token_each(dtype, dim, heads, kh):
    rrs, torch = _rrs()
    cache = _cache(rrs, torch, LENGTHS, kh, dim, 16, dtype, dim + heads)
    for most in (None, 1000):  # split by the table's width, and by the longest request
        _check(rrs, torch, cache, dtype, [1] * len(LENGTHS), LENGTHS, heads, ragged=False, max_length=most)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,heads,kh", [(64, 8, 8), (64, 32, 2), (128, 12, 4), (128, 24, 1), (256, 8, 2)])
@pytest.mark.parametrize("window", [0, 1, 16, 37, 500])
@pytest.mark.parametrize("page,layout", [(16, "tokens"), (128, "heads"), (32, "both")])
def test_drafts_and_windows(dtype, dim, heads, kh, window, page, layout):
    rrs, torch = _rrs()
    new = [1, 4, 0, 7, 2, 8, 3, 1]
    lengths = [1, 4, 3, 200, 33, 900, 515, 64]
    cache = _cache(rrs, torch, lengths, kh, dim, page, dtype, dim + window, layout)
    _check(rrs, torch, cache, dtype, new, lengths, heads, lead=3, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_drafts(dtype):
    """32 tokens of 24 queries a key head: several row blocks."""
    rrs, torch = _rrs()
    for dim in (64, 128, 256):
        lengths = [32, 300, 31 + 1024]
        cache = _cache(rrs, torch, lengths, 2, dim, 64, dtype, dim)
        _check(rrs, torch, cache, dtype, [32, 32, 31], lengths, 48, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long(dtype):
    """One request far into a context, split over its length; one and several key heads."""
    rrs, torch = _rrs()
    for kh, heads, n, page in ((1, 8, 70001, 1024), (4, 4, 33333, 16)):
        cache = _cache(rrs, torch, [n], kh, 64, page, dtype, 5)
        _check(rrs, torch, cache, dtype, [1], [n], heads, ragged=False)
        _check(rrs, torch, cache, dtype, [3], [n], heads, window=4001)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Weights that leave one key, a maximum that grows along the cache, and falling ones."""
    rrs, torch = _rrs()
    lengths = [1500, 1500, 1500]
    cache = _cache(rrs, torch, lengths, 1, 128, 16, dtype, 6)
    for b, ramp in enumerate((torch.linspace(-3, 3, 1500), torch.linspace(3, -3, 1500), torch.zeros(1500))):
        j = torch.arange(1500, device="cuda")
        number = cache.table[b].long()[j // 16]
        cache.k[number, j % 16, 0] = (cache.k[number, j % 16, 0].float() * 0.1 + ramp.cuda()[:, None]).to(cache.k.dtype)
    q = torch.ones(3, 4, 128, device="cuda").to(cache.k.dtype)
    _check(rrs, torch, cache, dtype, [1, 1, 1], lengths, 4, ragged=False, scale=0.25, q=q)
    _check(rrs, torch, cache, dtype, [1, 1, 1], lengths, 4, ragged=False, scale=-0.25, q=q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_stays_away(dtype, value):
    """Slots behind a request's end, missing pages, keys before the window and behind a row's own position hold
    anything: rows that do not see them are what they are without."""
    rrs, torch = _rrs()
    new, lengths = [3, 1, 5, 2], [40, 100, 333, 700]
    cache = _cache(rrs, torch, lengths, 2, 128, 16, dtype, 8)
    clean = rrs.Cache(cache.k.clone(), cache.v.clone(), cache.table)
    for pool in (cache.k, cache.v):
        keep = torch.zeros(pool.shape[:2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(lengths):
            j = torch.arange(max(0, n - new[b] + 1 - 37), n, device="cuda")  # a window of 37 from the first row on
            keep[cache.table[b].long()[j // 16], j % 16] = True
        pool[~keep] = value
    o, lse = _check(rrs, torch, cache, dtype, new, lengths, 8, window=37)
    o2, lse2 = _check(rrs, torch, clean, dtype, new, lengths, 8, window=37)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # the last drafted token's key and value: only its own row sees them
    for b, n in enumerate(lengths):
        number, slot = int(cache.table[b, (n - 1) // 16]), (n - 1) % 16
        cache.v[number, slot] = value
        if value == value:
            cache.v[number, slot, :, 1::2] = 1.0
    q = torch.randn(sum(new) + 2, 8, 128, generator=_gen(torch, 1), device="cuda").to(cache.k.dtype)
    got, gl = torch.full_like(q, 7.0), torch.empty(len(q), 8, device="cuda")
    rrs.seed_decode_attend(cache, _i32(torch, lengths), q, got, offsets=_offsets(torch, new), max_tokens=5, window=37, lse=gl)
    at = 0
    for m in new:
        assert torch.equal(got[at:at + m - 1], o[at:at + m - 1])
        assert not torch.isfinite(got[at + m - 1][:, 0::2].float()).any()
        at += m
    assert torch.equal(gl[:sum(new)], lse[:sum(new)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_visible_infinities(dtype):
    """Keys whose scores are minus infinity weigh nothing, plus infinity and NaN give NaN to the rows that see them, a row
    of nothing but minus infinity gets 0."""
    rrs, torch = _rrs()
    cache = _cache(rrs, torch, [300, 300, 300, 300], 1, 64, 16, dtype, 3)
    q = torch.ones(4, 2, 64, device="cuda").to(cache.k.dtype)
    q[:, 1] = -1
    inf = float("inf")

    def put(b, at, x):
        at = torch.as_tensor(at, device="cuda")
        cache.k[cache.table[b].long()[at // 16], at % 16] = x

    put(0, list(range(0, 300, 3)), -inf)
    put(1, [150], inf)
    put(2, [7], float("nan"))
    put(3, list(range(300)), -inf)
    o, lse = torch.empty_like(q), torch.empty(4, 2, device="cuda")
    for most in (300, 304):
        rrs.seed_decode_attend(cache, _i32(torch, [300] * 4), q, o, max_length=most, lse=lse)
        K, V = _gather(cache, 0, 300)
        want, wl, mag, _ = ref.attend(_np(q[0, :1]), _np(K[:, 0]), _np(V[:, 0]), np.array([299]), 0.125)
        _close(_np(o[0, :1]), want, HALF[dtype] * np.abs(want) + mag * 2.0 ** -14)
        assert torch.isnan(o[0, 1]).all() and torch.isnan(o[1, 0]).all() and torch.isfinite(o[1, 1].float()).all()
        assert torch.isnan(o[2]).all() and torch.isnan(lse[2]).all()
        assert (o[3, 0] == 0).all() and lse[3, 0] == -inf and torch.isnan(o[3, 1]).all()


def test_rows_that_see_nothing():
    """Empty requests, lengths below the new rows, missing pages throughout: zeros and minus infinity."""
    rrs, torch = _rrs()
    for dtype in ("bf16", "f32"):
        cache = _cache(rrs, torch, [64, 64, 64, 64, 2000], 2, 64, 16, dtype, 2)
        cache.table[3, :] = -1
        cache.table[2, 1:3] = 10 ** 6
        cache.table[4, 5:100] = -7
        o, lse = _check(rrs, torch, cache, dtype, [1, 3, 2, 2, 1], [0, 2, 64, 64, 2000], 4, max_length=2000)
        assert (o[0] == 0).all() and (lse[0] == -float("inf")).all() and (o[1] == 0).all() and (o[6:8] == 0).all()
        assert (lse[6:8] == -float("inf")).all() and torch.isfinite(lse[2:6]).all()
        _check(rrs, torch, cache, dtype, [1, 3, 2, 2, 1], [-5, -(1 << 31), 64, 64, 2000], 4)


def test_limits_of_the_call():
    """Lengths beyond max_length are cut, requests with more rows than max_tokens keep their rows behind."""
    rrs, torch = _rrs()
    cache = _cache(rrs, torch, [500, 500, 500], 2, 128, 16, "bf16", 2)
    _check(rrs, torch, cache, "bf16", [2, 1, 3], [500, (1 << 31) - 1, 120], 4, max_length=300)
    _check(rrs, torch, cache, "bf16", [2, 9, 3], [500, 400, 120], 4, most=2)
    q = torch.randn(6, 4, 128, device="cuda").bfloat16()
    for offsets in ([4, 2, 9, 1], [-3, 1, 100, 1 << 30], [0, 0, 0, 0], [6, 6, 6, 6], [-(1 << 31), (1 << 31) - 1, 3, 5]):
        o = torch.full_like(q, 7.0)
        rrs.seed_decode_attend(cache, _i32(torch, [500, 500, 500]), q, o, offsets=_i32(torch, offsets), max_tokens=4)
        torch.cuda.synchronize()
        assert torch.isfinite(o.float()).all()


@pytest.mark.parametrize("batch", [65, 256, 300, 600])
@pytest.mark.parametrize("most", [1, 6])
def test_many_requests(batch, most):
    """Shares that begin in any request: most short or empty, a few long, some without new rows."""
    rrs, torch = _rrs()
    r = np.random.default_rng(batch + most)
    new = [int(x) for x in r.integers(0, most + 1, batch)]
    new[0] = most
    lengths = [n + int(x) for n, x in zip(new, r.integers(0, 40, batch))]
    for b in (1, batch // 2, batch - 1):
        lengths[b] = 2000 + b
    cache = _cache(rrs, torch, lengths, 2, 64, 16, "bf16", batch)
    cache = rrs.Cache(cache.k, cache.v, torch.nn.functional.pad(cache.table, (0, 1024 - cache.table.shape[1]), value=-1))  # a far limit
    assert rrs.seed_attend_workspace_bytes(cache, sum(new), 6, max_tokens=most, ragged=True) > 0
    _check(rrs, torch, cache, "bf16", new, lengths, 6, lead=1)
    for b in range(batch):  # only the last one has rows, and only the first
        if b != batch - 1:
            new[b] = 0
    _check(rrs, torch, cache, "bf16", new[:-1] + [most], lengths, 6)
    _check(rrs, torch, cache, "bf16", [most] + [0] * (batch - 1), [max(lengths[0], most)] + lengths[1:], 6)
    _check(rrs, torch, cache, "bf16", [0] * batch, lengths, 6)


@pytest.mark.parametrize("most", [1, 4])
def test_offsets_beyond_32_bits(most):
    """Pages that lie more than 2^32 values behind the pool's start, stored to and read."""
    rrs, torch = _rrs()
    kh, heads, dim, page, stride = 2, 16, 128, 16, (1 << 32) // 2 + 64 * 8
    size = 3 * stride + page * kh * dim
    if torch.cuda.mem_get_info()[0] < 5 * size:  # keys and values of 2 bytes, and room
        pytest.skip("memory")
    pools = [torch.empty(size, dtype=torch.bfloat16, device="cuda").as_strided((4, page, kh, dim), (stride, kh * dim, dim, 1)) for _ in range(2)]
    table = _i32(torch, [[2, 0, 3, 1]])
    cache = rrs.Cache(*pools, table)
    n, g = 57, _gen(torch, 6)
    k, v = (torch.randn(n, kh, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    rrs.seed_cache_append(cache, _i32(torch, [n]), k, v, offsets=_offsets(torch, [n]))
    got_k, got_v = _gather(cache, 0, n)
    assert torch.equal(got_k, k) and torch.equal(got_v, v)
    _check(rrs, torch, cache, "bf16", [most], [n], heads)


def test_a_refused_call_leaves_no_trace():
    """A scale of 0 is refused; the same call with another one runs."""
    rrs, torch = _rrs()
    cache = _cache(rrs, torch, [9000], 2, 128, 16, "bf16", 2)
    q = torch.randn(1, 8, 128, device="cuda").bfloat16()
    o = torch.full_like(q, 7.0)
    with pytest.raises(rrs.SeedError):
        rrs.seed_decode_attend(cache, _i32(torch, [9000]), q, o, scale=0.0)
    assert (o == 7.0).all()
    _check(rrs, torch, cache, "bf16", [1], [9000], 8, ragged=False, q=q)


def test_strided_rows_and_workspace():
    """q and o as column ranges of wider rows, a workspace of the caller's, another stream: the same bits."""
    rrs, torch = _rrs()
    lengths, new = [5000, 4000], [1, 2]
    cache = _cache(rrs, torch, lengths, 2, 128, 16, "bf16", 12)
    need = rrs.seed_attend_workspace_bytes(cache, 3, 8, max_tokens=2, ragged=True)
    assert need > 0
    wide = torch.randn(3, 20, 128, device="cuda").bfloat16()
    q = wide[:, 4:12]
    args = (cache, _i32(torch, lengths))
    off = _offsets(torch, new)
    want = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    rrs.seed_decode_attend(*args, q.contiguous(), want, offsets=off, max_tokens=2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(wide, 7.0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    rrs.seed_decode_attend(*args, q, out[:, 12:], offsets=off, max_tokens=2, ws=ws, stream=stream)
    stream.synchronize()
    assert torch.equal(out[:, 12:], want) and (out[:, :12] == 7.0).all()
    rrs.seed_decode_attend(*args, q, out[:, 12:], offsets=off, max_tokens=2, stream=stream.cuda_stream)
    stream.synchronize()
    assert torch.equal(out[:, 12:], want)
    with pytest.raises(rrs.SeedError):
        rrs.seed_decode_attend(*args, q, want, offsets=off, max_tokens=2, ws=ws[:need - 16])


def test_graph_replays():
    """A token's calls in a graph, replayed over growing lengths with eager work between: each replay equals the
    eager result."""
    rrs, torch = _rrs()
    dt, kh, heads, dim, page = torch.bfloat16, 2, 8, 128, 16
    lengths = _i32(torch, [100, 1, 2047])
    a = _cache(rrs, torch, [2100] * 3, kh, dim, page, "bf16", 1)
    b = rrs.Cache(a.k.clone(), a.v.clone(), a.table)
    rotary = rrs.make_rotary(dim)
    q, k, v = (torch.zeros(3, n, dim, dtype=dt, device="cuda") for n in (heads, kh, kh))
    qo, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(3, heads, device="cuda")

    def step(cache, qo, o, lse):
        rrs.seed_cache_append(cache, lengths, k, v, rotary=rotary, q=q, q_out=qo)
        rrs.seed_decode_attend(cache, lengths, qo, o, lse=lse)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(a, qo, o, lse)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(a, qo, o, lse)
    g = _gen(torch, 4)
    for i in range(6):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        lengths += 1
        graph.replay()
        torch.cuda.synchronize()
        want, wl, wq = torch.empty_like(o), torch.empty_like(lse), torch.empty_like(q)
        step(b, wq, want, wl)
        torch.cuda.synchronize()
        b.k.copy_(a.k)  # the slot of the warm-up's first token
        b.v.copy_(a.v)
        if i > 0:
            assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(qo, wq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("share,most", [(5, 3), (7, 4), (6, 8), (11, 7)])
@pytest.mark.parametrize("lengths", [[97, 30, 100], [1999, 33, 700]])
@pytest.mark.parametrize("window", [0, 45])
def test_row_counts(dtype, dim, share, most, lengths, window):
    """Up to 16, 32, 64 and more rows of a key head, over caches that stay whole and that are cut: a page that is not
    there, NaN wherever no row looks, and an infinity that only its own column shows."""
    rrs, torch = _rrs()
    new, heads = [most, 1, most - 1], 2 * share
    cache = _cache(rrs, torch, lengths, 2, dim, 16, dtype, dim + share)
    cache.table[2, 1] = -1
    cache.table[0, (lengths[0] - most - 20) // 16] = 1 << 20
    clean = rrs.Cache(cache.k.clone(), cache.v.clone(), cache.table)
    keep = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        j = torch.arange(max(0, n - new[b] + 1 - window) if window else 0, n, device="cuda")
        number = cache.table[b].long()[j // 16]
        there = (number >= 0) & (number < len(cache.k))
        keep[number[there], j[there] % 16] = True
    cache.k[~keep] = float("nan")
    cache.v[~keep] = float("nan")
    o, lse = _check(rrs, torch, cache, dtype, new, lengths, heads, lead=1, window=window)
    o2, lse2 = _check(rrs, torch, clean, dtype, new, lengths, heads, lead=1, window=window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # the last but one position of the first request, key head 1: its last two tokens' rows see it
    at = lengths[0] - 2
    cache.v[int(cache.table[0, at // 16]), at % 16, 1, dim - 3] = float("inf")
    q = torch.randn(1 + sum(new) + 2, heads, dim, generator=_gen(torch, 1), device="cuda").to(cache.k.dtype)
    got = torch.full_like(q, 7.0)
    rrs.seed_decode_attend(cache, _i32(torch, lengths), q, got, offsets=_offsets(torch, new, 1), max_tokens=most, window=window)
    rows = slice(1 + most - 2, 1 + most)
    assert (got[rows, share:, dim - 3] == float("inf")).all()
    got[rows, share:, dim - 3] = o[rows, share:, dim - 3]
    assert torch.equal(got, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("share,most", [(4, 6), (8, 6)])
def test_large_scores_of_drafts(dtype, share, most):
    """A maximum that grows along the cache, and a falling one, over wavefronts that share tiles."""
    rrs, torch = _rrs()
    lengths = [1500, 1500]
    for dim in (64, 128, 256):
        cache = _cache(rrs, torch, lengths, 1, dim, 16, dtype, 6)
        for b, ramp in enumerate((torch.linspace(-3, 3, 1500), torch.linspace(3, -3, 1500))):
            j = torch.arange(1500, device="cuda")
            number = cache.table[b].long()[j // 16]
            cache.k[number, j % 16, 0] = (cache.k[number, j % 16, 0].float() * 0.1 + ramp.cuda()[:, None]).to(cache.k.dtype)
        q = torch.ones(2 * most + 2, share, dim, device="cuda").to(cache.k.dtype)
        _check(rrs, torch, cache, dtype, [most, most], lengths, share, scale=0.25, q=q)
        _check(rrs, torch, cache, dtype, [most, most], lengths, share, scale=-0.25, q=q)


def test_two_streams_and_graphs_of_drafts():
    """Two batches' drafts at once on two streams, each with a workspace of its own, and both captured and replayed over
    growing lengths: the bits of the calls one by one."""
    rrs, torch = _rrs()
    new, heads, dim = [6, 0, 3, 5], 16, 128
    off, most = _offsets(torch, new), 6
    sets = []
    for i, lengths in enumerate(([5000, 40, 3, 9000], [64, 7000, 2100, 300])):
        cache = _cache(rrs, torch, [n + 100 for n in lengths], 2, dim, 16, "bf16", 20 + i)
        q = torch.randn(sum(new), heads, dim, generator=_gen(torch, i), device="cuda").bfloat16()
        need = rrs.seed_attend_workspace_bytes(cache, sum(new), heads, max_tokens=most, ragged=True)
        sets.append(dict(cache=cache, lengths=_i32(torch, lengths), q=q, ws=torch.empty(need, dtype=torch.uint8, device="cuda"),
                         o=torch.empty_like(q), lse=torch.empty(sum(new), heads, device="cuda"), stream=torch.cuda.Stream()))

    def call(s, **kw):
        rrs.seed_decode_attend(s["cache"], s["lengths"], s["q"], s["o"], offsets=off, max_tokens=most, lse=s["lse"], **kw)

    def results():
        torch.cuda.synchronize()
        return [(s["o"].clone(), s["lse"].clone()) for s in sets]

    graphs = []
    for s in sets:
        call(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s["stream"]):
            call(s, ws=s["ws"])
        graphs.append(g)
    for turn in range(5):
        for s in sets:
            s["lengths"] += 7
            s["q"].normal_()
            call(s)
        want = results()
        for s in sets:
            s["o"].fill_(3.0)
            s["stream"].wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            for s in sets:
                call(s, ws=s["ws"], stream=s["stream"])
        got = results()
        for s in sets:
            s["o"].fill_(3.0)
        torch.cuda.synchronize()
        for s, g in zip(sets, graphs):
            with torch.cuda.stream(s["stream"]):
                g.replay()
        again = results()
        for a, b, c in zip(want, got, again):
            assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


def test_parts_of_a_context_join_by_lse():
    """Two halves of a context, attended apart and joined by their lse, are the whole."""
    rrs, torch = _rrs()
    cache = _cache(rrs, torch, [1024], 2, 64, 64, "f32", 3)
    q = torch.randn(1, 8, 64, device="cuda")
    whole, lse = torch.empty_like(q), torch.empty(1, 8, device="cuda")
    rrs.seed_decode_attend(cache, _i32(torch, [1024]), q, whole, lse=lse)
    parts = []
    for half in (slice(0, 8), slice(8, 16)):
        c = rrs.Cache(cache.k, cache.v, cache.table[:, half].contiguous())
        o, ls = torch.empty_like(q), torch.empty_like(lse)
        rrs.seed_decode_attend(c, _i32(torch, [512]), q, o, lse=ls)
        parts.append((o, ls))
    w = torch.softmax(torch.stack([p[1] for p in parts]), 0)[..., None]
    joined = w[0] * parts[0][0] + w[1] * parts[1][0]
    assert (joined - whole).abs().max() < 2.0 ** -18
    assert (torch.logaddexp(parts[0][1], parts[1][1]) - lse).abs().max() < 2.0 ** -18
