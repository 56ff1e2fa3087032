"""GPU tests of the prompt path (seed_prefill_conv, seed_decode_conv, seed_prefill_scan,
seed_norm_rows) against the plain fp64 forms of prompt_ref.py, which receive exactly the values the
device buffers hold.

Tolerances, element by element. A value rounded once to its format is off by at most half a step,
eps / 2 of its size (bf16 2^-8, fp32 2^-24). Before that rounding:
  - convolution: at most 5 fp32 operations per output, each off by 2^-24 of the sum of absolute
    terms, through an activation of slope at most 1.1 whose own evaluation is good to 2^-20 (bf16)
    or 2^-22 (fp32): 2^-18 and 2^-20 of that sum;
  - norm: the mean square of positive terms and its root are good to (8 + log2 dim) 2^-24, the sum
    x + s skip to 2^-24 of its absolute terms, the gate as above: 2^-18 and 2^-19 of the scale;
  - scan states: one fp32 rounding per token and element and sums of up to 128 products; over T
    tokens the roundings add like a random walk, sqrt(T) 2^-24 times a small factor: 1e-5 of
    |S|_F for T up to 4096 (the package's fp32 tolerance);
  - scan read-outs: the state's error and a d_k-long sum, 1e-5 |S|_F |q|, and where matrix
    instructions take operands in two 16-bit pieces, 2^-16 |S|_F |q| more: 3e-5 in all.
"""
from __future__ import annotations

import numpy as np
import pytest

import prompt_ref as ref

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


def _code(rrs, name):
    return {"bf16": rrs.SEED_BF16, "f32": rrs.SEED_F32}[name]


def _np(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def _gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _offsets(torch, lens, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _close(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off; worst {np.abs(got - want).max():.3e} at {np.argwhere(bad)[0]}"


# ---- convolution ----------------------------------------------------------------------------------

LENS = {
    "one": [1],
    "short": [0, 1, 2, 3, 0, 4, 5, 0],
    "edges": [16, 15, 17, 1, 31, 33, 0, 2],
    "long": [129, 0, 513],
    "all-empty": [0, 0, 0],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("channels", [8, 77, 2056])
def test_prefill_conv(dtype, width, lens, channels):
    rrs, torch = _rrs()
    L = LENS[lens]
    n = sum(L)
    g = _gen(torch, width * 100 + channels)
    dt = _dt(torch, dtype)
    for with_window, bias, act in ((True, True, True), (False, False, False)):
        lead, tail = 3, 5  # rows around the sequences stay as they are
        x = torch.randn(n + lead + tail, channels, device="cuda", generator=g).to(dt)
        x[:lead] = float("nan")
        x[lead + n:] = float("nan")
        w = torch.randn(width, channels, device="cuda", generator=g)
        b = torch.randn(channels, device="cuda", generator=g) if bias else None
        win = torch.randn(len(L), width - 1, channels, device="cuda", generator=g).to(dt) if with_window else None
        y = torch.full_like(x, 7.0)
        out = torch.full((len(L), width - 1, channels), 9.0, dtype=dt, device="cuda")
        conv = rrs.make_conv(len(L), channels, width, _code(rrs, dtype), silu=act)
        rrs.seed_prefill_conv(conv, x, _offsets(torch, L, lead), w, b, out, y, window_in=win)
        torch.cuda.synchronize()
        yr, wr, mag = ref.conv(_np(x[lead:lead + n]), L, _np(w), _np(b), _np(win), act)
        _close(_np(y[lead:lead + n]), yr, HALF[dtype] * np.abs(yr) + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -20) * mag)
        assert np.array_equal(_np(out), wr)
        assert (y[:lead] == 7.0).all() and (y[lead + n:] == 7.0).all()


def test_prefill_conv_in_pieces_equals_one_pass():
    """A prompt convolved in three calls through its windows is the prompt convolved in one."""
    rrs, torch = _rrs()
    g = _gen(torch, 5)
    ch, cuts = 264, [[20, 1], [1, 0], [30, 40]]
    x = [torch.randn(sum(c[b] for c in cuts), ch, device="cuda", generator=g).bfloat16() for b in range(2)]
    w = torch.randn(4, ch, device="cuda", generator=g)
    conv = rrs.make_conv(2, ch, 4)
    whole = torch.cat(x)
    yw, ww = torch.empty_like(whole), torch.empty(2, 3, ch, dtype=torch.bfloat16, device="cuda")
    rrs.seed_prefill_conv(conv, whole, _offsets(torch, [len(t) for t in x]), w, None, ww, yw)
    at, win, parts = [0, 0], None, [[], []]
    for c in cuts:
        piece = torch.cat([x[b][at[b]:at[b] + c[b]] for b in range(2)])
        y, nw = torch.empty_like(piece), torch.empty_like(ww)
        rrs.seed_prefill_conv(conv, piece, _offsets(torch, c), w, None, nw, y, window_in=win)
        parts[0].append(y[:c[0]])
        parts[1].append(y[c[0]:])
        at, win = [at[0] + c[0], at[1] + c[1]], nw
    assert torch.equal(torch.cat(parts[0] + parts[1]), yw) and torch.equal(win, ww)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,channels,width", [(1, 8, 2), (1, 77, 4), (9, 4096, 4), (130, 264, 3), (33, 1, 4)])
def test_decode_conv(dtype, batch, channels, width):
    rrs, torch = _rrs()
    g = _gen(torch, batch + channels)
    dt = _dt(torch, dtype)
    x = torch.randn(batch, channels, device="cuda", generator=g).to(dt)
    w = torch.randn(width, channels, device="cuda", generator=g)
    b = torch.randn(channels, device="cuda", generator=g)
    win = torch.randn(batch, width - 1, channels, device="cuda", generator=g).to(dt)
    active = (torch.rand(batch, device="cuda", generator=g) < 0.7).to(torch.uint8)
    conv = rrs.make_conv(batch, channels, width, _code(rrs, dtype))
    yr, wr, mag = ref.conv(_np(x), [1] * batch, _np(w), _np(b), _np(win), True)
    tol = HALF[dtype] * np.abs(yr) + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -20) * mag
    y, out = torch.full_like(x, 7.0), torch.full_like(win, 9.0)
    rrs.seed_decode_conv(conv, x, w, b, win, y, window_out=out)
    _close(_np(y), yr, tol)
    assert np.array_equal(_np(out), wr)
    # masked, the window in place, y over x
    y2, win2, on = x.clone(), win.clone(), _np(active) != 0
    rrs.seed_decode_conv(conv, y2, w, b, win2, y2, active=active)
    _close(_np(y2)[on], yr[on], tol[on])
    assert np.array_equal(_np(win2)[on], wr[on])
    assert np.array_equal(_np(y2)[~on], _np(x)[~on]) and np.array_equal(_np(win2)[~on], _np(win)[~on])


def test_conv_strided_columns_and_far_rows():
    """Rows that are columns of a wider buffer whose byte offsets pass 2^32, for prompts and tokens."""
    rrs, torch = _rrs()
    g = _gen(torch, 3)
    n, stride, ch = 40000, 65536, 64  # 5.2 GB of bf16
    buf = torch.empty(n, stride, dtype=torch.bfloat16, device="cuda")
    x, y = buf[:, 128:128 + ch], buf[:, 256:256 + ch]
    x.copy_(torch.randn(n, ch, device="cuda", generator=g))
    buf[:, 256 + ch:256 + ch + 8] = 3.0
    w = torch.randn(4, ch, device="cuda", generator=g)
    lens = [17000, 3, 22997]
    out = torch.empty(3, 3, ch, dtype=torch.bfloat16, device="cuda")
    rrs.seed_prefill_conv(rrs.make_conv(3, ch, 4), x, _offsets(torch, lens), w, None, out, y)
    dense = torch.empty(n, ch, dtype=torch.bfloat16, device="cuda")
    out2 = torch.empty_like(out)
    rrs.seed_prefill_conv(rrs.make_conv(3, ch, 4), x.contiguous(), _offsets(torch, lens), w, None, out2, dense)
    assert torch.equal(y, dense) and torch.equal(out, out2)
    assert (buf[:, 256 + ch:256 + ch + 8] == 3.0).all()
    tail = slice(n - 40, n)
    yr, _, mag = ref.conv(_np(x[n - 43:]), [43], _np(w), None, None, True)
    _close(_np(y[tail]), yr[3:], HALF["bf16"] * np.abs(yr[3:]) + 2.0 ** -18 * mag[3:])


# ---- scan -----------------------------------------------------------------------------------------

SCAN_LENS = {
    "one": [1],
    "ragged": [0, 1, 2, 5, 63, 64, 65, 0, 130, 17],
    "long": [700, 3, 257],
}


def _scan_inputs(torch, g, kind, n, heads, kh, dk, dv, dtype, scale=1.0):
    dt = _dt(torch, dtype)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=g)

    q, k = normal(n, kh, dk), normal(n, kh, dk)
    if kind != ref.MAMBA2:
        q, k = torch.nn.functional.normalize(q, dim=-1), torch.nn.functional.normalize(k, dim=-1)
    beta = torch.rand(n, heads, device="cuda", generator=g)
    gate = 1 - 0.1 * torch.rand(*((n, heads, dk) if kind == ref.KDA else (n, heads)), device="cuda", generator=g)
    return q.to(dt), k.to(dt), (scale * normal(n, heads, dv)).to(dt), beta, gate


def _check_scan(got_o, got_S, want, dtype):
    o, S, mag = want
    _close(got_o, o, HALF[dtype] * np.abs(o) + 3e-5 * mag[:, :, None])
    top = np.sqrt((S * S).sum((2, 3)))
    err = np.sqrt(((got_S - S) ** 2).sum((2, 3)))
    assert (err <= 1e-5 * top + 1e-30).all(), f"state off by {np.max(err / np.maximum(top, 1e-30)):.3e}"


def _run_scan(rrs, torch, kind, lens, t, S0, dims, dtype, S=None, **kw):
    heads, dk, dv = dims
    q, k, v, beta, gate = t
    shape = rrs.make_shape(kind, len(lens), heads, dk, dv, 8, 8, _code(rrs, dtype))
    S = torch.full((len(lens), heads, dk, dv), 5.0, device="cuda") if S is None else S
    o = torch.full((q.shape[0], heads, dv), 7.0, dtype=v.dtype, device="cuda")
    rrs.seed_prefill_scan(shape, kw.pop("offsets", _offsets(torch, lens)), q, k, v, beta, gate, S, o, S0=S0, **kw)
    return o, S


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("lens", list(SCAN_LENS))
def test_scan(kind, dtype, dk, dv, lens):
    rrs, torch = _rrs()
    L = SCAN_LENS[lens]
    for heads, kh, carry in ((3, 1, True), (4, 2, False)):
        g = _gen(torch, 1000 * kind + dk + dv + heads)
        t = _scan_inputs(torch, g, kind, sum(L), heads, kh, dk, dv, dtype)
        S0 = torch.randn(len(L), heads, dk, dv, device="cuda", generator=g) if carry else None
        o, S = _run_scan(rrs, torch, kind, L, t, S0, (heads, dk, dv), dtype)
        torch.cuda.synchronize()
        _check_scan(_np(o), _np(S), ref.scan(kind, L, *map(_np, t), _np(S0)), dtype)


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("batch,heads,most", [(90, 4, 5), (130, 8, 3), (70, 16, 40)])
def test_scan_of_many_units(kind, dtype, dk, dv, batch, heads, most):
    """Many requests, of a few tokens each and of more."""
    rrs, torch = _rrs()
    r = np.random.default_rng(batch + most)
    lens = r.integers(0, most + 1, batch).tolist()
    g = _gen(torch, batch)
    t = _scan_inputs(torch, g, kind, sum(lens), heads, heads, dk, dv, dtype)
    S0 = torch.randn(batch, heads, dk, dv, device="cuda", generator=g)
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, (heads, dk, dv), dtype)
    _check_scan(_np(o), _np(S), ref.scan(kind, lens, *map(_np, t), _np(S0)), dtype)


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_gates_of_every_size(kind, dtype):
    """Gates of 1, of 0, so small that their product underflows, and strong ones token after token,
    next to beta of 0 and 1 and the same key again and again."""
    rrs, torch = _rrs()
    lens, heads, dk, dv = [150, 70, 66], 2, 128, 64
    g = _gen(torch, 17)
    q, k, v, beta, gate = _scan_inputs(torch, g, kind, sum(lens), heads, 2, dk, dv, dtype)
    gate[:150] = 1.0
    gate[20], gate[64], gate[65], gate[127] = 0.0, 0.0, 0.0, 0.0
    gate[100:104] = 1e-30
    gate[150:220] = torch.exp(-12.0 * torch.rand(gate[150:220].shape, device="cuda", generator=g))
    gate[180:190] = 1e-42  # below the smallest normal fp32 value
    beta[30:60], beta[60:75] = 0.0, 1.0
    k[40:120] = k[40].clone()
    t = (q, k, v, beta, gate)
    S0 = torch.randn(3, heads, dk, dv, device="cuda", generator=g)
    o, S = _run_scan(rrs, torch, kind, lens, t, S0, (heads, dk, dv), dtype)
    _check_scan(_np(o), _np(S), ref.scan(kind, lens, *map(_np, t), _np(S0)), dtype)


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_scan_values_of_every_size(kind, scale):
    rrs, torch = _rrs()
    lens, heads, dk, dv = [90, 140], 2, 64, 128
    t = _scan_inputs(torch, _gen(torch, 23), kind, sum(lens), heads, 1, dk, dv, "bf16", scale)
    o, S = _run_scan(rrs, torch, kind, lens, t, None, (heads, dk, dv), "bf16")
    _check_scan(_np(o), _np(S), ref.scan(kind, lens, *map(_np, t), None), "bf16")


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_in_place_and_in_pieces(kind, dtype):
    """States updated in place, a prompt continued over calls; sequences that get no tokens keep
    their states to the bit."""
    rrs, torch = _rrs()
    heads, dk, dv = 2, 128, 128
    g = _gen(torch, 31)
    whole = [130, 200]
    t = _scan_inputs(torch, g, kind, sum(whole), heads, 2, dk, dv, dtype)
    want = ref.scan(kind, whole, *map(_np, t), None)
    S = torch.zeros(2, heads, dk, dv, device="cuda")
    outs, at = [[], []], [0, 130]
    for cut in ([100, 0], [29, 64], [0, 135], [1, 1]):
        idx = torch.cat([torch.arange(at[b], at[b] + cut[b]) for b in range(2)]).cuda()
        before = S.clone()
        o, _ = _run_scan(rrs, torch, kind, cut, tuple(x[idx] for x in t), S, (heads, dk, dv), dtype, S=S)
        for b in range(2):
            if cut[b] == 0:
                assert torch.equal(S[b], before[b])
            at[b] += cut[b]
        outs[0].append(o[:cut[0]])
        outs[1].append(o[cut[0]:])
    _check_scan(_np(torch.cat(outs[0] + outs[1])), _np(S), want, dtype)


@pytest.mark.parametrize("kind", [ref.GDN, ref.KDA, ref.MAMBA2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_neighbours(kind, dtype):
    """NaN and infinities of one sequence, and of rows outside every sequence, stay there; rows
    outside are not written; q, k and v are column ranges of one wide buffer."""
    rrs, torch = _rrs()
    lens, heads, kh, dk, dv, lead, tail = [70, 33, 90], 2, 1, 64, 64, 9, 13
    n = sum(lens)
    g = _gen(torch, 41)
    q, k, v, beta, gate = _scan_inputs(torch, g, kind, n, heads, kh, dk, dv, dtype)
    S0 = torch.randn(3, heads, dk, dv, device="cuda", generator=g)
    want = ref.scan(kind, lens, *map(_np, (q, k, v, beta, gate)), _np(S0))
    rows = lead + n + tail
    buf = torch.full((rows, kh * dk * 2 + heads * dv + 16), float("nan"), dtype=q.dtype, device="cuda")
    wide = (buf[:, :kh * dk].view(rows, kh, dk), buf[:, kh * dk:2 * kh * dk].view(rows, kh, dk),
            buf[:, 2 * kh * dk:2 * kh * dk + heads * dv].view(rows, heads, dv))
    wb = torch.full((rows, heads), float("nan"), device="cuda")
    wg = torch.full((rows,) + gate.shape[1:], float("nan"), device="cuda")
    for dst, src in zip(wide + (wb, wg), (q, k, v, beta, gate)):
        dst[lead:lead + n] = src
    mid = slice(lead + 70, lead + 103)
    wide[2][mid] = float("inf")
    wide[1][lead + 80] = float("nan")
    o, S = _run_scan(rrs, torch, kind, lens, wide + (wb, wg), S0, (heads, dk, dv), dtype, offsets=_offsets(torch, lens, lead))
    assert (o[:lead] == 7.0).all() and (o[lead + n:] == 7.0).all()
    keep = np.r_[0:70, 103:n]
    _check_scan(_np(o[lead:lead + n])[keep], _np(S)[[0, 2]], tuple(x[i] for x, i in zip(want, (keep, [0, 2], keep))), dtype)
    assert not torch.isfinite(S[1]).all()


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("carry", [False, True])
def test_scan_of_few_long_prompts(kind, dk, dv, carry):
    """Prompts long and few enough to be cut into segments (equal and ragged ones, with empty and
    short sequences between), the states in place."""
    rrs, torch = _rrs()
    for lens in ([2600], [5000, 0, 1], [2100, 6000, 40, 2500]):
        heads = 2
        g = _gen(torch, dk + dv + len(lens))
        t = _scan_inputs(torch, g, kind, sum(lens), heads, 1, dk, dv, "bf16")
        S0 = torch.randn(len(lens), heads, dk, dv, device="cuda", generator=g) if carry else None
        want = ref.scan(kind, lens, *map(_np, t), _np(S0))
        o, S = _run_scan(rrs, torch, kind, lens, t, S0, (heads, dk, dv), "bf16", S=S0)
        _check_scan(_np(o), _np(S), want, "bf16")


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
@pytest.mark.parametrize("where", [5, 40, 1500, 2999])
def test_scan_is_causal_for_values_that_are_not_finite(kind, where):
    """What is not finite at a token leaves the read-outs before it as they were, in the token's own
    chunk and segment too: v and k, beta and the gate in turn."""
    rrs, torch = _rrs()
    heads, dk, dv, n = 1, 128, 64, 3000
    t = _scan_inputs(torch, _gen(torch, 47), kind, n, heads, 1, dk, dv, "bf16")
    want, _, mag = ref.scan(kind, [n], *map(_np, t), None)
    for which, value in ((2, float("inf")), (1, float("nan")), (3, float("inf")), (4, float("nan")), (2, float("nan"))):
        bad = [x.clone() for x in t]
        bad[which][where] = value
        o, S = _run_scan(rrs, torch, kind, [n], tuple(bad), None, (heads, dk, dv), "bf16")
        got = _np(o[:where])
        _close(got, want[:where], HALF["bf16"] * np.abs(want[:where]) + 3e-5 * mag[:where, :, None])
        assert not torch.isfinite(S).all()


@pytest.mark.parametrize("log_stride", [23, 24])
def test_scan_rows_far_apart(log_stride):
    """Rows whose byte offsets pass 2^32, at a stride that chunks still take and at one they do not."""
    rrs, torch = _rrs()
    heads, dk, dv, n, stride = 1, 64, 64, 200, 1 << log_stride
    t = _scan_inputs(torch, _gen(torch, 59), ref.GDN, n, heads, 1, dk, dv, "bf16")
    buf = torch.empty((n - 1) * stride + 4 * 64, dtype=torch.bfloat16, device="cuda")
    far = [buf.as_strided((n, 1, 64), (stride, 64, 1), 64 * i) for i in range(4)]
    for dst, src in zip(far, t[:3]):
        dst.copy_(src)
    shape = rrs.make_shape(rrs.SEED_GDN, 2, heads, dk, dv, 8, 8, rrs.SEED_BF16)
    S = torch.empty(2, heads, dk, dv, device="cuda")
    rrs.seed_prefill_scan(shape, _offsets(torch, [77, 123]), *far[:3], t[3], t[4], S, far[3])
    _check_scan(_np(far[3]), _np(S), ref.scan(ref.GDN, [77, 123], *map(_np, t), None), "bf16")


def test_long_scan_captured_and_replayed():
    """A prompt cut into segments, in a graph whose workspace comes from torch's allocator."""
    rrs, torch = _rrs()
    heads, d, n = 1, 64, 2700
    t = _scan_inputs(torch, _gen(torch, 61), ref.GDN, n, heads, 1, d, d, "bf16")
    shape = rrs.make_shape(rrs.SEED_GDN, 1, heads, d, d, 8, 8, rrs.SEED_BF16)
    off = _offsets(torch, [n])

    def run(o, S):
        rrs.seed_prefill_scan(shape, off, *t, S, o)

    eager, graphed = ([torch.empty(n, heads, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, heads, d, d, device="cuda")]
                      for _ in range(2))
    run(*graphed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*graphed)
    for i in range(4):
        t[2].copy_(torch.randn(n, heads, d, device="cuda", generator=_gen(torch, i)))
        graph.replay()
        torch.cuda.synchronize()
        run(*eager)
        torch.cuda.synchronize()
        assert torch.equal(eager[0], graphed[0]) and torch.equal(eager[1], graphed[1])


def test_long_scan_with_wrong_offsets_and_on_given_streams():
    """Cut prompts whose offsets decrease or leave the buffer stay inside it and leave the rows around
    alone; the call's own workspace follows the stream it is given."""
    rrs, torch = _rrs()
    heads, d, n = 2, 64, 5000
    t = _scan_inputs(torch, _gen(torch, 67), ref.GDN, n, heads, 1, d, d, "bf16")
    guard = torch.full((n + 64, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    shape = rrs.make_shape(rrs.SEED_GDN, 4, heads, d, d, 8, 8, rrs.SEED_BF16)
    room = torch.full((6, heads, d, d), 3.0, device="cuda")
    off = torch.tensor([0, n, -7, n, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert rrs.seed_prefill_workspace_bytes(shape, rrs.seed_prompt(4 * n, None, 1, d, d, 2 * d, 2 * d)) > 0
    rrs.seed_prefill_scan(rrs.make_shape(rrs.SEED_GDN, 4, heads, d, d, 8, 8, rrs.SEED_BF16), off, *t, room[1:5], guard[32:32 + n])
    torch.cuda.synchronize()
    assert (guard[:32] == 7.0).all() and (guard[32 + n:] == 7.0).all()
    assert (room[0] == 3.0).all() and (room[5] == 3.0).all()
    o0, S0 = _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, d, d), "bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        o1, S1 = _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, d, d), "bf16", stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(S0, S1) and torch.equal(o0, o1)


def test_scan_workspaces():
    """A given workspace, one of torch's allocator, and one that is too small or misaligned."""
    rrs, torch = _rrs()
    heads, dk, dv, n = 1, 64, 64, 2600
    t = _scan_inputs(torch, _gen(torch, 53), ref.GDN, n, heads, 1, dk, dv, "bf16")
    shape = rrs.make_shape(rrs.SEED_GDN, 1, heads, dk, dv, 8, 8, rrs.SEED_BF16)
    need = rrs.seed_prefill_workspace_bytes(shape, rrs.seed_prompt(n, None, 1, dk, dk, dv, dv))
    assert need > 0
    assert rrs.seed_prefill_workspace_bytes(shape, rrs.seed_prompt(64, None, 1, dk, dk, dv, dv)) == 0
    o0, S0 = _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, dk, dv), "bf16")
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    o1, S1 = _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, dk, dv), "bf16", ws=ws[:need])
    assert torch.equal(o0, o1) and torch.equal(S0, S1) and (ws[need:] == 255).all()
    with pytest.raises(rrs.SeedError) as e:
        _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, dk, dv), "bf16", ws=ws[:need - 1])
    assert e.value.status == rrs.SEED_ERR_WORKSPACE
    with pytest.raises(rrs.SeedError) as e:
        _run_scan(rrs, torch, ref.GDN, [n], t, None, (heads, dk, dv), "bf16", ws=ws[1:need + 1])
    assert e.value.status == rrs.SEED_ERR_ARG


def test_scan_wrong_offsets_stay_inside():
    """Offsets that decrease or leave the buffer give clamped sequences and touch nothing else."""
    rrs, torch = _rrs()
    heads, dk, dv, n = 2, 64, 64, 80
    t = _scan_inputs(torch, _gen(torch, 43), ref.GDN, n, heads, 2, dk, dv, "bf16")
    off = torch.tensor([-5, 30, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    o, S = _run_scan(rrs, torch, ref.GDN, [0] * 3, t, None, (heads, dk, dv), "bf16", offsets=off)
    torch.cuda.synchronize()
    first = ref.scan(ref.GDN, [30], *(_np(x[:30]) for x in t), None)
    assert np.abs(_np(S[0]) - first[1][0]).max() < 1e-4 and (S[1] == 0).all()
    x = torch.randn(n, 64, device="cuda").bfloat16()
    y, win = torch.full_like(x, 7.0), torch.empty(3, 3, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(4, 64, device="cuda")
    rrs.seed_prefill_conv(rrs.make_conv(3, 64, 4), x, off, w, None, win, y)
    torch.cuda.synchronize()
    assert torch.isfinite(y.float()).all() and (win[1] == 0).all()


# ---- norm -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,heads,dim", [(1, 32, 128), (7, 3, 64), (5, 2, 200), (3, 5, 77), (130, 1, 512), (9, 1, 1),
                                            (4, 1, 2048), (3, 2, 4104), (2, 1, 8192), (2, 1, 16392), (1, 1, 9001), (0, 2, 64)])
def test_norm_rows(dtype, rows, heads, dim):
    rrs, torch = _rrs()
    g = _gen(torch, rows + dim)
    dt = _dt(torch, dtype)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)

    x, z, sk = (r(rows, heads, dim).to(dt) for _ in range(3))
    w, sc = 1 + 0.2 * r(heads, dim), r(heads)
    for gate, first, skip, scale, total in ((None, False, None, None, False), (z, False, sk, sc, True), (z, True, sk, None, False),
                                            (z, True, None, None, True), (None, False, sk, sc, True)):
        y = torch.full_like(x, 7.0)
        tt = torch.full_like(x, 7.0) if total else None
        rrs.seed_norm_rows(x, w, y, gate=gate, eps=1e-5, gate_first=first, skip=skip, skip_scale=scale, total=tt)
        yr, tr, mag = ref.norm_rows(_np(x), _np(w), _np(gate), 1e-5, first, _np(skip), _np(scale))
        _close(_np(y), yr, HALF[dtype] * np.abs(yr) + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -19) * mag)
        if total:
            _close(_np(tt), tr, HALF[dtype] * np.abs(tr) + 2.0 ** -23 * (np.abs(_np(x)) + (0 if skip is None else np.abs(tr - _np(x)))))


def test_norm_rows_in_place_and_strided():
    rrs, torch = _rrs()
    g = _gen(torch, 71)
    rows, heads, dim = 37, 4, 64
    buf = torch.randn(rows, 3 * heads * dim + 24, device="cuda", generator=g).bfloat16()
    x, z, res = (buf[:, i * heads * dim:(i + 1) * heads * dim].view(rows, heads, dim) for i in range(3))
    w, sc = torch.randn(heads, dim, device="cuda", generator=g), torch.randn(heads, device="cuda", generator=g)
    args = dict(gate=z.contiguous(), skip=res.contiguous(), skip_scale=sc)
    y0, t0 = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda")
    rrs.seed_norm_rows(x.contiguous(), w, y0, total=t0, **args)
    rest = buf[:, 3 * heads * dim:].clone()
    rrs.seed_norm_rows(x, w, x, gate=z, skip=res, skip_scale=sc, total=res)  # y over x, the sum over the stream
    assert torch.equal(x, y0) and torch.equal(res, t0) and torch.equal(buf[:, 3 * heads * dim:], rest)


def test_norm_rows_of_zeros_and_infinities():
    """A row of zeros gives zeros; an infinite or NaN value stays in its group."""
    rrs, torch = _rrs()
    x = torch.ones(3, 4, 64, device="cuda")
    x[0] = 0
    x[1, 2, 5] = float("inf")
    x[2, 1, 63] = float("nan")
    y = torch.empty_like(x)
    rrs.seed_norm_rows(x, torch.ones(4, 64, device="cuda"), y, eps=1e-6)
    assert (y[0] == 0).all()
    good = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    good[0] = good[1, 2] = good[2, 1] = False
    assert torch.allclose(y[good], torch.ones_like(y[good]), rtol=0, atol=1e-6)
    assert torch.isnan(y[1, 2, 5]) and torch.isnan(y[2, 1]).all()


# ---- streams, graphs, the path together -----------------------------------------------------------

def test_prompt_path_on_another_stream_and_in_a_graph():
    """The three prompt operators captured once and replayed on new contents, next to eager work."""
    rrs, torch = _rrs()
    g = _gen(torch, 81)
    lens, heads, dk, dv = [100, 0, 61], 2, 128, 64
    n, ch = sum(lens), 2 * heads * dk + heads * dv
    off = _offsets(torch, lens)
    conv = rrs.make_conv(3, ch, 4)
    shape = rrs.make_shape(rrs.SEED_MAMBA2, 3, heads, dk, dv, 8, 8, rrs.SEED_BF16)
    w = torch.randn(4, ch, device="cuda", generator=g) * 0.4
    nw = torch.ones(heads, dv, device="cuda")
    x = torch.randn(n, ch, device="cuda", generator=g).bfloat16()
    beta, gate = torch.rand(n, heads, device="cuda", generator=g), torch.rand(n, heads, device="cuda", generator=g)

    def buffers():
        return dict(y=torch.empty_like(x), win=torch.empty(3, 3, ch, dtype=torch.bfloat16, device="cuda"),
                    S=torch.empty(3, heads, dk, dv, device="cuda"),
                    o=torch.empty(n, heads, dv, dtype=torch.bfloat16, device="cuda"))

    def layer(d, stream=None):
        rrs.seed_prefill_conv(conv, x, off, w, None, d["win"], d["y"], stream=stream)
        q, k = (d["y"][:, i * heads * dk:(i + 1) * heads * dk].view(n, heads, dk) for i in range(2))
        v = d["y"][:, 2 * heads * dk:].view(n, heads, dv)
        rrs.seed_prefill_scan(shape, off, q, k, v, beta, gate, d["S"], d["o"], stream=stream)
        rrs.seed_norm_rows(d["o"], nw, d["o"], gate=v, stream=stream)

    eager, graphed = buffers(), buffers()
    layer(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer(graphed)
    side.synchronize()
    assert all(torch.equal(eager[k], graphed[k]) for k in eager)
    other = buffers()
    layer(other, stream=side)
    side.synchronize()
    assert all(torch.equal(eager[k], other[k]) for k in eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(graphed)
    for _ in range(4):
        x.copy_(torch.randn(n, ch, device="cuda", generator=g))
        gate.copy_(torch.rand(n, heads, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        layer(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(eager[k], graphed[k]) for k in eager)


@pytest.mark.parametrize("kind", [ref.GDN, ref.MAMBA2])
def test_a_layer_from_prompt_to_token(kind):
    """One layer's prompt (residual norm, convolution, scan, gated read-out norm), its states
    compressed, then tokens (convolution, decode step, norm), each stage against fp64 on the values
    it was given."""
    rrs, torch = _rrs()
    g = _gen(torch, 91)
    lens, heads, dk, dv, width, rank = [70, 1, 40], 2, 64, 64, 256, 16
    n, B = sum(lens), len(lens)
    ch = 2 * heads * dk + heads * dv
    off = _offsets(torch, lens)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)

    block, stream = r(n, 1, width).bfloat16(), r(n, 1, width).bfloat16()
    w_in, proj = 1 + 0.1 * r(1, width), r(width, ch) / width ** 0.5
    filt, w_out = 0.5 * r(4, ch), 1 + 0.1 * r(heads, dv)
    conv = rrs.make_conv(B, ch, 4)
    shape = rrs.make_shape(kind, B, heads, dk, dv, rank, 8, rrs.SEED_BF16)

    def split(y):
        m = y.shape[0]
        q, k = (y[:, i * heads * dk:(i + 1) * heads * dk].view(m, heads, dk) for i in range(2))
        return q, k, y[:, 2 * heads * dk:].view(m, heads, dv)

    # prompt
    h = torch.empty_like(block)
    before = _np(stream)
    rrs.seed_norm_rows(block, w_in, h, skip=stream, total=stream)
    yr, tr, mag = ref.norm_rows(_np(block), _np(w_in), None, 1e-6, False, before, None)
    _close(_np(h), yr, HALF["bf16"] * np.abs(yr) + 2.0 ** -18 * mag)
    _close(_np(stream), tr, HALF["bf16"] * np.abs(tr) + 2.0 ** -22 * (np.abs(_np(block)) + np.abs(before)))
    x = (h.view(n, width).float() @ proj).bfloat16()
    y, win = torch.empty_like(x), torch.empty(B, 3, ch, dtype=torch.bfloat16, device="cuda")
    rrs.seed_prefill_conv(conv, x, off, filt, None, win, y)
    q, k, v = split(y)
    beta = 0.05 * torch.rand(n, heads, device="cuda", generator=g)
    gate = 1 - 0.1 * torch.rand(n, heads, device="cuda", generator=g)
    S = torch.empty(B, heads, dk, dv, device="cuda")
    o = torch.empty(n, heads, dv, dtype=torch.bfloat16, device="cuda")
    rrs.seed_prefill_scan(shape, off, q, k, v, beta, gate, S, o)
    _check_scan(_np(o), _np(S), ref.scan(kind, lens, *map(_np, (q, k, v, beta, gate)), None), "bf16")
    out = torch.empty_like(o)
    rrs.seed_norm_rows(o, w_out, out, gate=v)
    yr, _, mag = ref.norm_rows(_np(o), _np(w_out), _np(v), 1e-6, False, None, None)
    _close(_np(out), yr, HALF["bf16"] * np.abs(yr) + 2.0 ** -18 * mag)
    # the states leave the prefill; the dense form goes on beside the factored one
    vbar = torch.nn.functional.normalize(r(heads, dv), dim=-1)
    st = rrs.State.empty(shape)
    rrs.seed_state_from_dense(shape, S.view(B * heads, dk, dv), vbar, st)
    for step in range(4):
        xt = r(B, ch).bfloat16()
        yt = torch.empty_like(xt)
        yr, wr, mag = ref.conv(_np(xt), [1] * B, _np(filt), None, _np(win), True)
        rrs.seed_decode_conv(conv, xt, filt, None, win, yt)
        _close(_np(yt), yr, HALF["bf16"] * np.abs(yr) + 2.0 ** -18 * mag)
        assert np.array_equal(_np(win), wr)
        qt, kt, vt = (t.contiguous() for t in split(yt))
        bt = 0.05 * torch.rand(B, heads, device="cuda", generator=g)
        gt = 1 - 0.1 * torch.rand(B, heads, device="cuda", generator=g)
        # a prompt of one token is the dense decode step
        dense, od = S.clone(), torch.empty(B, heads, dv, dtype=torch.bfloat16, device="cuda")
        rrs.seed_dense_decode_step(shape, dense, qt, kt, vt, bt, gt, od)
        ot = torch.empty_like(od)
        rrs.seed_prefill_scan(shape, _offsets(torch, [1] * B), qt, kt, vt, bt, gt, S, ot, S0=S)
        assert (dense - S).norm() <= 1e-5 * dense.norm()
        of = torch.empty_like(od)
        rrs.seed_decode_step(shape, st, rank + step, qt, kt, vt, bt, gt, vbar, of)
        on = torch.empty_like(od)
        rrs.seed_norm_rows(of, w_out, on, gate=vt)
        yr, _, mag = ref.norm_rows(_np(of), _np(w_out), _np(vt), 1e-6, False, None, None)
        _close(_np(on), yr, HALF["bf16"] * np.abs(yr) + 2.0 ** -18 * mag)
