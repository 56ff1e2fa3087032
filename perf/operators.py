"""Performance cases of the prompt path and the token path of a recurrent layer.

A GDN, KDA or Mamba-2 layer serves a prompt as: short causal convolution over the projected
channels, the gated scan that builds each head's state (handed to seed_state_from_dense
afterwards), and the head norm of the read-outs; and a token as the same convolution on its
window, the decode step, and the norm. The cases below stand for these operators at the head
shapes and channel counts of the package's own workloads (synth/): 16, 32 or 64 heads with
d_k = 128 and d_v = 128 or 64, prompts of up to 8192 tokens, batches of up to 512 requests.

    conv   seed_prefill_conv   y_t = act(bias + sum_j w_j x_{t - width + 1 + j}) over packed prompts
    step   seed_decode_conv    the same for one token per request, from the request's window
    scan   seed_prefill_scan   S_t = G_t S_{t-1} + beta_t k_t (v_t - [delta] (G_t S_{t-1})^T k_t)^T,
                               o_t = S_t^T q_t over packed prompts, from and to fp32 states
    norm   seed_norm_rows      w * x / sqrt(mean x^2 + eps), x = o + s * skip, with a SiLU gate

`own` selects the package's kernels; otherwise run() computes the operators from elementary
torch operations. exact() evaluates the definitions token after token in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per block of the plain scan
EPS = 1e-6


# ---- the cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one request's token: 16 key heads and 32 value heads of 128 as q | k | v channels; the
        # smallest launch there is, where only latency counts
        dict(name="conv-token-one", op="step", batch=1, channels=8192, width=4, dtype="bf16", silu=True, bias=True),
        # a full decode batch with key heads of its own for every head
        dict(name="conv-token-batch", op="step", batch=512, channels=12288, width=4, dtype="bf16", silu=True, bias=False),
        # a prefill batch of requests of unequal length, continuing earlier chunks of their prompts
        dict(name="conv-prompts", op="conv", batch=16, tokens=32768, channels=8192, width=4, dtype="bf16", silu=True,
             bias=True, carry=True, ragged=True),
        # odd everything: fp32, three taps, no activation, a channel count that fills no vector
        dict(name="conv-odd-f32", op="conv", batch=5, tokens=3001, channels=1037, width=3, dtype="f32", silu=False,
             bias=False, carry=False, ragged=True),
        # one long prompt of a GDN layer with 16 key heads: few units, many tokens
        dict(name="scan-gdn-one-long", op="scan", kind="gdn", batch=1, tokens=8192, heads=32, key_heads=16, d_k=128,
             d_v=128, dtype="bf16", carry=False, ragged=False),
        # a prefill batch of GDN prompts of unequal length, continuing from earlier states
        dict(name="scan-gdn-prompts", op="scan", kind="gdn", batch=16, tokens=32768, heads=32, key_heads=32, d_k=128,
             d_v=128, dtype="bf16", carry=True, ragged=True),
        # a few drafted tokens for each of many requests: the states' own traffic
        dict(name="scan-gdn-few-tokens", op="scan", kind="gdn", batch=128, tokens=300, heads=16, key_heads=16, d_k=128,
             d_v=128, dtype="bf16", carry=True, ragged=True),
        # one Mamba-2 prompt, one B / C group for all heads
        dict(name="scan-mamba2-one", op="scan", kind="mamba2", batch=1, tokens=2048, heads=64, key_heads=1, d_k=128,
             d_v=64, dtype="bf16", carry=False, ragged=False),
        # a prefill batch of Mamba-2 prompts, 8 groups
        dict(name="scan-mamba2-prompts", op="scan", kind="mamba2", batch=16, tokens=32768, heads=64, key_heads=8,
             d_k=128, d_v=64, dtype="bf16", carry=True, ragged=True),
        # short KDA prompts: a gate for every key channel
        dict(name="scan-kda-prompts", op="scan", kind="kda", batch=8, tokens=2500, heads=32, key_heads=32, d_k=128,
             d_v=128, dtype="bf16", carry=False, ragged=True),
        # the read-out norm of one token, gated
        dict(name="norm-token", op="norm", rows=1, heads=32, d=128, dtype="bf16", gate="after", skip=False, total=False),
        # the read-out norm of a prefill batch: Mamba-2's D skip, gate before the norm
        dict(name="norm-prompts", op="norm", rows=32768, heads=64, d=64, dtype="bf16", gate="first", skip=True,
             total=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "conv", "scan", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        return dict(op="step", batch=_log(rng, 1, 512), channels=_log(rng, 256, 12288), width=rng.randint(2, 4), dtype=dtype,
                    silu=rng.random() < 0.7, bias=rng.random() < 0.5)
    if op == "conv":
        batch = _log(rng, 1, 64)
        return dict(op="conv", batch=batch, tokens=_log(rng, max(8, batch), 16384), channels=_log(rng, 256, 8192),
                    width=rng.randint(2, 4), dtype=dtype, silu=rng.random() < 0.7, bias=rng.random() < 0.5,
                    carry=rng.random() < 0.5, ragged=True)
    if op == "norm":
        if rng.random() < 0.4:  # the norm before a block: a residual stream, its sum written too
            return dict(op="norm", rows=_log(rng, 1, 8192), heads=1, d=8 * _log(rng, 64, 1024), dtype=dtype, gate="none",
                        skip=True, total=True)
        return dict(op="norm", rows=_log(rng, 1, 16384), heads=rng.choice([4, 16, 24, 32, 64]), d=rng.choice([64, 128]),
                    dtype=dtype, gate=rng.choice(["none", "after", "first"]), skip=rng.random() < 0.5, total=False)
    kind = rng.choice(["gdn", "gdn", "mamba2", "mamba2", "kda"])
    batch = _log(rng, 1, 64)
    heads = rng.choice([1, 4, 6, 16, 24, 32])
    shared = rng.choice([h for h in (1, 2, 4) if heads % h == 0])
    # the sequential forms (fp32, per-channel gates) are drawn at the prompt lengths that suit them
    most = 16384 if dtype == "bf16" and kind != "kda" else 4096
    longest = 4096 if dtype == "bf16" and kind != "kda" else 1024
    tokens = min(_log(rng, max(2, batch), most), batch * longest // 2)
    return dict(op="scan", kind=kind, batch=batch, tokens=tokens, heads=heads, key_heads=heads // shared,
                d_k=rng.choice([64, 128, 128]), d_v=rng.choice([64, 128]), dtype=dtype, carry=rng.random() < 0.5, ragged=True)


def _lengths(case):
    """The requests' lengths: a property of the case. Ragged ones lie within about a factor of six;
    with many requests one is empty and one a single token."""
    n, total = case["batch"], case["tokens"]
    if not case["ragged"] or n == 1:
        return [total // n + (1 if i < total % n else 0) for i in range(n)]
    r = random.Random(1000003 * n + total)
    w = [r.uniform(0.3, 1.7) for _ in range(n)]
    if n >= 4:
        w[1], w[2] = 0.0, 0.0
    lens = [int(total * x / sum(w)) for x in w]
    if n >= 4 and total > n:
        lens[2] = 1
    left, i = total - sum(lens), 0
    while left != 0:  # what the rounding left, over the others in turn
        j = i % n
        if not (n >= 4 and j in (1, 2)) and lens[j] + (1 if left > 0 else -1) >= 0:
            lens[j] += 1 if left > 0 else -1
            left += -1 if left > 0 else 1
        i += 1
    return lens


# ---- inputs ---------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case=case)
    op = case["op"]
    if op in ("step", "conv"):
        c, width = case["channels"], case["width"]
        rows = case["batch"] if op == "step" else case["tokens"]
        s["x"] = normal(rows, c).to(dt)
        s["weight"] = normal(width, c) * 0.5
        s["bias"] = normal(c) * 0.1 if case["bias"] else None
        s["window"] = normal(case["batch"], width - 1, c).to(dt) if op == "step" or case["carry"] else None
        s["window_out"] = torch.empty(case["batch"], width - 1, c, dtype=dt, device=dev)
        s["y"] = torch.empty_like(s["x"])
    elif op == "norm":
        rows, heads, d = case["rows"], case["heads"], case["d"]
        s["x"] = normal(rows, heads, d).to(dt)
        s["weight"] = 1.0 + 0.1 * normal(heads, d)
        s["gate"] = normal(rows, heads, d).to(dt) if case["gate"] != "none" else None
        s["skip"] = normal(rows, heads, d).to(dt) if case["skip"] else None
        s["skip_scale"] = uniform(0.2, 1.5, heads) if case["skip"] else None
        s["total"] = torch.empty_like(s["x"]) if case["total"] else None
        s["y"] = torch.empty_like(s["x"])
    else:
        n, b, heads, kh = case["tokens"], case["batch"], case["heads"], case["key_heads"]
        dk, dv = case["d_k"], case["d_v"]
        q, k = normal(n, kh, dk), normal(n, kh, dk)
        if case["kind"] != "mamba2":  # queries and keys of unit length, as the delta rule has them
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        s["q"], s["k"] = q.to(dt), k.to(dt)
        s["v"] = (normal(n, heads, dv) + 0.5 * normal(heads, dv)).to(dt)
        if case["kind"] == "mamba2":  # step sizes from 0.001 to 0.1 by head, input-dependent around them
            step = torch.exp(uniform(math.log(1e-3), math.log(0.1), heads))
            dtime = torch.nn.functional.softplus(normal(n, heads) + torch.log(torch.expm1(step)))
            s["beta"], s["g"] = dtime, torch.exp(-dtime * uniform(1.0, 16.0, heads))
        else:
            s["beta"] = uniform(0.0, 1.0, n, heads)
            s["g"] = uniform(0.9, 1.0, n, heads, dk) if case["kind"] == "kda" else uniform(0.9, 1.0, n, heads)
        s["S0"] = 0.3 * normal(b, heads, dk, dv) if case["carry"] else None
        s["S"] = torch.empty(b, heads, dk, dv, device=dev)
        s["o"] = torch.empty(n, heads, dv, dtype=dt, device=dev)
    if op in ("conv", "scan"):
        s["lengths"] = _lengths(case)
        ends = torch.tensor([0] + s["lengths"]).cumsum(0)
        s["offsets"] = ends.to(torch.int32).to(dev)
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import rank_recurrent_state_amd as rrs
        io = rrs.SEED_BF16 if c["dtype"] == "bf16" else rrs.SEED_F32
        if c["op"] == "step":
            conv = rrs.make_conv(c["batch"], c["channels"], c["width"], io, silu=c["silu"])
            rrs.seed_decode_conv(conv, s["x"], s["weight"], s["bias"], s["window"], s["y"], window_out=s["window_out"])
            return {"y": s["y"], "window": s["window_out"]}
        if c["op"] == "conv":
            conv = rrs.make_conv(c["batch"], c["channels"], c["width"], io, silu=c["silu"])
            rrs.seed_prefill_conv(conv, s["x"], s["offsets"], s["weight"], s["bias"], s["window_out"], s["y"],
                                  window_in=s["window"])
            return {"y": s["y"], "window": s["window_out"]}
        if c["op"] == "norm":
            rrs.seed_norm_rows(s["x"], s["weight"], s["y"], gate=s["gate"], eps=EPS, gate_first=c["gate"] == "first",
                               skip=s["skip"], skip_scale=s["skip_scale"], total=s["total"])
            return {"y": s["y"], "total": s["total"]} if c["total"] else {"y": s["y"]}
        kind = {"gdn": rrs.SEED_GDN, "kda": rrs.SEED_KDA, "mamba2": rrs.SEED_MAMBA2}[c["kind"]]
        shape = rrs.make_shape(kind, c["batch"], c["heads"], c["d_k"], c["d_v"], 16, 16, io)
        rrs.seed_prefill_scan(shape, s["offsets"], s["q"], s["k"], s["v"], s["beta"], s["g"], s["S"], s["o"], S0=s["S0"])
        return {"o": s["o"], "S": s["S"]}
    if c["op"] == "step":
        return _plain_step(s)
    if c["op"] == "conv":
        return _plain_conv(s)
    if c["op"] == "norm":
        return _plain_norm(s)
    return _plain_scan(s)


def _act(y, c):
    return y / (1 + torch.exp(-y)) if c["silu"] else y


def _plain_step(s):
    c, x = s["case"], s["x"].float()
    taps = torch.cat([s["window"].float(), x[:, None]], 1)  # [batch, width, channels]
    y = (taps * s["weight"]).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": _act(y, c).to(s["x"].dtype), "window": taps[:, 1:].to(s["x"].dtype)}


def _rows(s):
    """Each packed row's request and its place in it."""
    starts, n = s["offsets"].long(), s["case"]["tokens"]
    row = torch.arange(n, device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return row, seq, row - starts[seq]


def _plain_conv(s):
    c, x = s["case"], s["x"]
    width = c["width"]
    row, seq, pos = _rows(s)
    past = s["window"] if s["window"] is not None else torch.zeros_like(s["window_out"])
    y = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    if s["bias"] is not None:
        y += s["bias"]
    for j in range(width):
        at = row - (width - 1 - j)
        tap = torch.where((pos >= width - 1 - j)[:, None], x[at.clamp_min(0)], past[seq, (pos + j).clamp_max(width - 2)])
        y += tap.float() * s["weight"][j]
    # the last width - 1 inputs of every request, those of its old window where it is shorter
    starts = s["offsets"].long()
    i = torch.arange(width - 1, device=x.device)
    p = (starts[1:] - starts[:-1])[:, None] - (width - 1) + i  # place in the request, below 0 in the window
    got = x[(starts[:-1, None] + p).clamp(0, max(c["tokens"] - 1, 0))]
    old = torch.gather(past, 1, (p + width - 1).clamp(0, width - 2)[..., None].expand_as(past))
    return {"y": _act(y, c).to(x.dtype), "window": torch.where((p >= 0)[..., None], got, old)}


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    if s["skip"] is not None:
        x = x + s["skip_scale"][:, None] * s["skip"].float()
    out = {"total": x.to(s["x"].dtype)} if c["total"] else {}
    gate = None
    if s["gate"] is not None:
        z = s["gate"].float()
        gate = z / (1 + torch.exp(-z))
    if c["gate"] == "first":
        x = x * gate
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    if c["gate"] == "after":
        y = y * gate
    return {"y": y.to(s["x"].dtype), **out}


def _padded(s, multiple):
    """The packed rows as [batch, heads, length, ...] with idle tokens (g = 1, all else 0) behind."""
    c, b = s["case"], s["case"]["batch"]
    share = c["heads"] // c["key_heads"]
    length = max(-(-max(s["lengths"]) // multiple) * multiple, multiple)
    _, seq, pos = _rows(s)

    def pad(x, fill=0.0, repeat=1):
        full = torch.full((b, length) + x.shape[1:], fill, dtype=torch.float32, device=x.device)
        full[seq, pos] = x.float()
        full = full.transpose(1, 2)
        return full.repeat_interleave(repeat, 1) if repeat > 1 else full.contiguous()

    return (pad(s["q"], 0, share), pad(s["k"], 0, share), pad(s["v"]), pad(s["beta"]), pad(s["g"], 1.0), seq, pos, length)


def _plain_scan(s):
    c = s["case"]
    b, h, dk, dv = c["batch"], c["heads"], c["d_k"], c["d_v"]
    delta = c["kind"] != "mamba2"
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros_like(s["S"])
    if c["kind"] == "kda":  # a gate per key channel: token after token
        q, k, v, beta, g, seq, pos, length = _padded(s, 1)
        o = torch.empty_like(v)
        for t in range(length):
            S = S * g[:, :, t, :, None]
            kt = k[:, :, t, :, None]
            w = beta[:, :, t, None] * (v[:, :, t] - (S * kt).sum(2))
            S = S + kt * w[:, :, None]
            o[:, :, t] = (S * q[:, :, t, :, None]).sum(2)
        return {"o": o.transpose(1, 2)[seq, pos].to(s["o"].dtype), "S": S}
    # blocks of CHUNK tokens: the delta rule's residuals w solve (I + A) w = beta (v - e^c S^T k)
    q, k, v, beta, g, seq, pos, length = _padded(s, CHUNK)
    n = length // CHUNK
    q, k, v = (x.reshape(b, h, n, CHUNK, -1) for x in (q, k, v))
    beta = beta.reshape(b, h, n, CHUNK)
    # the gates' running products: 64 bits, since their logarithms are subtracted
    cum = torch.log(g.double().clamp_min(1e-60)).reshape(b, h, n, CHUNK).cumsum(-1)
    decay = torch.tril(torch.exp(torch.tril(cum[..., :, None] - cum[..., None, :]))).float()
    head, tail, whole = torch.exp(cum).float(), torch.exp(cum[..., -1:] - cum).float(), torch.exp(cum[..., -1]).float()
    mix = torch.matmul(q, k.transpose(-1, -2)) * decay
    if delta:
        A = torch.tril(torch.matmul(k, k.transpose(-1, -2)) * decay * beta[..., None], -1)
        T = torch.zeros_like(A)
        for t in range(CHUNK):  # forward substitution, every block at once
            T[..., t, :] = -torch.matmul(A[..., t, None, :t], T[..., :t, :])[..., 0, :]
            T[..., t, t] += 1
        T = T * beta[..., None, :]
    o = torch.empty_like(v)
    for i in range(n):
        if delta:
            w = torch.matmul(T[:, :, i], v[:, :, i] - head[:, :, i, :, None] * torch.matmul(k[:, :, i], S))
        else:
            w = beta[:, :, i, :, None] * v[:, :, i]
        o[:, :, i] = head[:, :, i, :, None] * torch.matmul(q[:, :, i], S) + torch.matmul(mix[:, :, i], w)
        S = whole[:, :, i, None, None] * S + torch.matmul(k[:, :, i].transpose(-1, -2), tail[:, :, i, :, None] * w)
    return {"o": o.reshape(b, h, length, dv).transpose(1, 2)[seq, pos].to(s["o"].dtype), "S": S}


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "step":
        cells = case["batch"] * case["channels"]
        per = case["channels"] * 4 * (case["width"] + (1 if case["bias"] else 0))
        return {"bytes": cells * e * (2 + 2 * (case["width"] - 1)) + per, "flops": cells * (2 * case["width"] + 4)}
    if op == "conv":
        cells = case["tokens"] * case["channels"]
        per = case["channels"] * 4 * (case["width"] + (1 if case["bias"] else 0))
        window = case["batch"] * case["channels"] * (case["width"] - 1) * e
        return {"bytes": 2 * cells * e + per + window * (2 if case["carry"] else 1), "flops": cells * (2 * case["width"] + 4)}
    if op == "norm":
        cells = case["rows"] * case["heads"] * case["d"]
        streams = 2 + (case["gate"] != "none") + case["skip"] + case["total"]
        return {"bytes": cells * e * streams + case["heads"] * case["d"] * 4, "flops": cells * 8}
    n, heads, dk, dv = case["tokens"], case["heads"], case["d_k"], case["d_v"]
    rows = n * (2 * case["key_heads"] * dk + 2 * heads * dv) * e
    scalars = 4 * n * heads * (1 + (dk if case["kind"] == "kda" else 1))
    states = 4 * case["batch"] * heads * dk * dv * (2 if case["carry"] else 1)
    return {"bytes": rows + scalars + states, "flops": n * heads * dk * dv * (4 if case["kind"] == "mamba2" else 6)}


# ---- the definitions, in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        if case["skip"]:
            x = x + s["skip_scale"].double().view(1, -1, 1) * s["skip"].double()
        out = {}
        if case["total"]:
            out["total"] = x
        silu = s["gate"].double() * torch.sigmoid(s["gate"].double()) if case["gate"] != "none" else None
        y = x * silu if case["gate"] == "first" else x
        y = s["weight"].double() * y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        return {"y": y * silu if case["gate"] == "after" else y, **out}
    if op in ("step", "conv"):
        width, c = case["width"], case["channels"]
        lens = [1] * case["batch"] if op == "step" else s["lengths"]
        ys, windows, at = [], [], 0
        for b, n in enumerate(lens):  # a request's old window and its inputs, one after the other
            past = s["window"][b].double() if s["window"] is not None else torch.zeros(width - 1, c, dtype=torch.float64, device="cuda")
            line = torch.cat([past, s["x"][at:at + n].double()])
            y = sum(line[j:j + n] * s["weight"][j].double() for j in range(width))
            if s["bias"] is not None:
                y = y + s["bias"].double()
            ys.append(y * torch.sigmoid(y) if case["silu"] else y)
            windows.append(line[n:])
            at += n
        return {"y": torch.cat(ys), "window": torch.stack(windows)}
    # the recurrence itself, all requests side by side, the ended ones left alone
    b, heads, dk, dv = case["batch"], case["heads"], case["d_k"], case["d_v"]
    lens = torch.tensor(s["lengths"], device="cuda")
    first = s["offsets"][:-1].long()
    of = torch.arange(heads, device="cuda") // (heads // case["key_heads"])
    S = s["S0"].double() if s["S0"] is not None else torch.zeros(b, heads, dk, dv, dtype=torch.float64, device="cuda")
    o = torch.zeros(case["tokens"], heads, dv, dtype=torch.float64, device="cuda")
    for t in range(max(s["lengths"])):
        live = torch.nonzero(lens > t)[:, 0]
        rows = first[live] + t
        at = slice(None) if len(live) == b else live
        k, q = s["k"][rows][:, of].double(), s["q"][rows][:, of].double()
        g = s["g"][rows].double()
        now = S[at] * (g[..., None] if case["kind"] == "kda" else g[..., None, None])
        w = s["v"][rows].double()
        if case["kind"] != "mamba2":
            w = w - torch.matmul(k[:, :, None, :], now)[:, :, 0]
        now += k[..., None] * (s["beta"][rows].double()[..., None] * w)[:, :, None]
        S[at] = now
        o[rows] = torch.matmul(q[:, :, None, :], now)[:, :, 0]
    return {"o": o, "S": S}
