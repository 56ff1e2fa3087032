"""Performance cases of the attention layers that a hybrid model has between its recurrent ones, and
of its drafted tokens.

Such a layer serves a token (or a few drafted ones) as: rotary positions on its queries and keys,
the keys and values stored into the pages of the request's cache, attention over that cache; and
behind the last layer the drafted tokens are checked against the model's probabilities. The cases
stand for these operators at the head sizes of the package's own workloads and their neighbours (64,
128 and 256), requests of one token to 131072, batches of up to 512 requests.

    rotate  seed_rotate_rows    pairs of a head turned by position * frequency
    append  seed_cache_append   the same for q and k, k and v stored at their place of a paged cache
    attend  seed_decode_attend  softmax(scale q K^T) V of each request's newest tokens over its pages
    verify  seed_verify_drafts  drafts kept while u q(x) < p(x), the next token drawn from max(p - q, 0)

`own` selects the package's kernels; otherwise run() computes the operators from elementary torch
operations. exact() evaluates the definitions in 64 bits, request after request.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------------------------

def listed():
    return [
        # queries and keys of a prefill batch, side by side in one buffer: the whole head in halves
        dict(name="rotate-prompts", op="rotate", rows=32768, heads=40, dim=128, rot=128, interleaved=False, scaling="none",
             far=8192, dtype="bf16"),
        # odd everything: fp32, 20 of 72 values in neighbouring pairs, positions of a stretched long context
        dict(name="rotate-odd-f32", op="rotate", rows=1001, heads=5, dim=72, rot=20, interleaved=True, scaling="parts",
             far=1000000, dtype="f32"),
        # one request's token: the smallest launch there is, where only latency counts
        dict(name="append-token-one", op="append", batch=1, tokens=1, history=700, heads=32, key_heads=8, dim=128, rot=128,
             interleaved=False, scaling="none", page=16, layout="tokens", dtype="bf16"),
        # a prefill batch of unequal prompts into an empty cache, a quarter of each head rotated
        dict(name="append-prompts", op="append", batch=16, tokens=32768, history=0, heads=16, key_heads=4, dim=256, rot=64,
             interleaved=False, scaling="none", page=64, layout="tokens", dtype="bf16"),
        # one request's token after a short prompt
        dict(name="attend-token-one", op="attend", batch=1, fresh=1, longest=700, heads=32, key_heads=8, dim=128, page=16,
             window=0, layout="tokens", dtype="bf16"),
        # one request far into a long context: the cache's length is the only axis to share out
        dict(name="attend-one-long", op="attend", batch=1, fresh=1, longest=131072, heads=32, key_heads=8, dim=128, page=64,
             window=0, layout="tokens", dtype="bf16"),
        # a decode batch of requests of unequal length
        dict(name="attend-batch", op="attend", batch=64, fresh=1, longest=16384, heads=64, key_heads=8, dim=128, page=16,
             window=0, layout="tokens", dtype="bf16"),
        # several drafted tokens per request, two key heads of 256 for all queries
        dict(name="attend-drafts", op="attend", batch=48, fresh=6, longest=8192, heads=16, key_heads=2, dim=256, page=32,
             window=0, layout="heads", dtype="bf16"),
        # odd everything: fp32, three queries a key head, a window that ends inside pages
        dict(name="attend-odd-f32", op="attend", batch=7, fresh=3, longest=5003, heads=12, key_heads=4, dim=64, page=16,
             window=1001, layout="tokens", dtype="f32"),
        # one request's few drafts
        dict(name="verify-one", op="verify", batch=1, drafts=4, vocab=32000, dtype="f32", sampled=True),
        # a decode batch of drafts from a smaller model, over an odd vocabulary
        dict(name="verify-batch", op="verify", batch=128, drafts=5, vocab=150001, dtype="f32", sampled=True),
        # drafts that come without probabilities (looked up in the prompt)
        dict(name="verify-lookup", op="verify", batch=200, drafts=8, vocab=65536, dtype="bf16", sampled=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend", "attend", "verify"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    turn = dict(interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "base", "parts"]))
    layout = rng.choice(["tokens", "tokens", "heads"])
    if op == "rotate":
        dim = rng.choice([64, 72, 80, 96, 128, 128, 256])
        return dict(op=op, rows=_log(rng, 1, 16384), heads=rng.choice([1, 5, 8, 24, 40]), dim=dim,
                    rot=rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]), far=_log(rng, 100, 1000000), dtype=dtype, **turn)
    key_heads, share = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16])
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 16, 32, 64, 256])
    heads = dict(heads=min(key_heads * share, 64 // key_heads * key_heads), key_heads=key_heads, dim=dim, page=page, layout=layout,
                 dtype=dtype)
    if op == "append":
        batch = _log(rng, 1, 256)
        return dict(op=op, batch=batch, tokens=_log(rng, batch, 16384), history=rng.choice([0, _log(rng, 1, 500)]),
                    rot=rng.choice([dim, dim // 4, 2 * rng.randint(1, dim // 2)]), **heads, **turn)
    if op == "attend":
        batch, longest = _log(rng, 1, 256), _log(rng, 1, 131072)
        most = 1 << 30  # bytes of K and V
        per = 2 * key_heads * dim * (2 if dtype == "bf16" else 4)
        longest = max(1, min(longest, most // (batch * per)))
        return dict(op=op, batch=batch, fresh=rng.choice([1, 1, 1, 2, 5, 8]), longest=longest,
                    window=rng.choice([0, 0, _log(rng, 16, 4096)]), **heads)
    batch, drafts = _log(rng, 1, 256), rng.randint(0, 8)
    return dict(op=op, batch=batch, drafts=drafts, vocab=min(_log(rng, 100, 262144), (1 << 27) // (batch * (drafts + 1))), dtype=dtype,
                sampled=rng.random() < 0.6)


def _rows_of(case):
    """The requests' new rows: a property of the case. Prompts lie within about a factor of six; among
    several drafting requests the counts run from one to the most."""
    n = case["batch"]
    r = random.Random(7919 * n + case.get("tokens", 0) + case.get("longest", 0) + case.get("vocab", 0))
    if case["op"] == "append":
        if n == case["tokens"]:
            return [1] * n
        w = [r.uniform(0.3, 1.7) for _ in range(n)]
        rows = [1 + int((case["tokens"] - n) * x / sum(w)) for x in w]
        rows[0] += case["tokens"] - sum(rows)
        return rows
    most = case["fresh"] if case["op"] == "attend" else case["drafts"] + 1
    return [most] + [r.randint(1, most) for _ in range(n - 1)]


def _lengths(case, rows):
    """Tokens in each request's cache, the new ones included: within a factor of eight, the first
    request the longest; of several one has no history."""
    n = case["batch"]
    r = random.Random(104729 * n + case.get("tokens", 0) + case.get("longest", 0))
    if case["op"] == "append":
        return [k + (r.randint(case["history"] // 2, case["history"]) if case["history"] else 0) for k in rows]
    top = case["longest"]
    lens = [top] + [_log(r, max(1, top // 8), top) for _ in range(n - 1)]
    if n >= 4:
        lens[2] = 1
    return [max(a, b) for a, b in zip(lens, rows)]


# ---- inputs ---------------------------------------------------------------------------------------

SCALINGS = {  # for contexts beyond the trained one; lengths in tokens, ramps in turns over the trained length
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "base": dict(base=10000.0, factor=8.0),
    "parts": dict(base=500000.0, factor=32.0, length=8192.0, low=1.0, high=32.0),
}


def _turns(case):
    """Turns per position of every pair, in 64 bits: a table of a few hundred bytes, kept like a weight."""
    kind, rot = case["scaling"], case["rot"]
    o = SCALINGS[kind]
    base = o["base"]
    if kind == "base" and rot > 2:
        base = base * o["factor"] ** (rot / (rot - 2))
    t = [base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
    if kind == "linear":
        t = [x / o["factor"] for x in t]
    if kind == "parts":
        keep = [min(max((o["length"] * x - o["low"]) / (o["high"] - o["low"]), 0.0), 1.0) for x in t]
        t = [x * (k + (1 - k) / o["factor"]) for x, k in zip(t, keep)]
    return t


def _amplitude(case):
    return 0.1 * math.log(SCALINGS["parts"]["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _handle(case):
    import rank_recurrent_state_amd as rrs
    kind = {"none": rrs.SEED_ROTARY_PLAIN, "linear": rrs.SEED_ROTARY_LINEAR, "base": rrs.SEED_ROTARY_BASE,
            "parts": rrs.SEED_ROTARY_PARTS}[case["scaling"]]
    return rrs.make_rotary(case["rot"], interleaved=case["interleaved"], scaling=kind, amplitude=_amplitude(case),
                           **SCALINGS[case["scaling"]])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=case)
    if op in ("rotate", "append"):
        s["turns"] = torch.tensor(_turns(case), dtype=torch.float64, device=dev)
        if own:
            s["rotary"] = _handle(case)
    if op == "rotate":
        s["x"] = normal(case["rows"], case["heads"], case["dim"]).to(dt)
        s["positions"] = torch.randint(0, case["far"], (case["rows"],), generator=gen, device=dev, dtype=torch.int32)
        s["y"] = torch.empty_like(s["x"])
        return s
    rows = _rows_of(case)
    n = sum(rows)
    s["rows"] = rows
    s["offsets"] = torch.tensor([0] + rows).cumsum(0).to(torch.int32).to(dev)
    if op == "verify":
        # logits of a spread that leaves some hundred likely tokens, the draft's close to the target's
        logits = 2.5 * normal(n, case["vocab"])
        s["target"] = torch.softmax(logits, -1).to(dt)
        noise = -torch.log(-torch.log(torch.rand(n, case["vocab"], generator=gen, device=dev).clamp(1e-9, 1 - 1e-7)))
        logits += 0.5 * normal(n, case["vocab"])
        s["draft"] = torch.softmax(logits, -1).to(dt) if case["sampled"] else None
        s["drafts"] = (logits + noise if case["sampled"] else logits).argmax(-1).to(torch.int32)  # sampled, or the likeliest
        s["uniforms"] = torch.rand(n, generator=gen, device=dev)
        s["draws"] = torch.rand(case["batch"], generator=gen, device=dev)
        s["tokens"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["counts"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
        return s
    lens, page, kh, dim = _lengths(case, rows), case["page"], case["key_heads"], case["dim"]
    s["length_list"] = lens
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    # pages in any order, as a pool that serves many requests hands them out; some stay unused
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=gen, device=dev)[:sum(need)].to(torch.int32)
    s["table"] = torch.zeros(case["batch"], max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        s["table"][b, :k] = order[at:at + k]
        at += k
    shape = (pool, page, kh, dim) if case["layout"] == "tokens" else (pool, kh, page, dim)
    for name in ("k_pages", "v_pages"):
        x = torch.empty(shape, dtype=dt, device=dev)
        for i in range(0, pool, 4096):  # in pieces: the fp32 normals of a large pool are twice its size
            x[i:i + 4096] = normal(*x[i:i + 4096].shape)
        s[name] = x if case["layout"] == "tokens" else x.transpose(1, 2)
    s["q"] = normal(n, case["heads"], dim).to(dt)
    if op == "append":
        s["k"], s["v"] = normal(n, kh, dim).to(dt), normal(n, kh, dim).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
    else:
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, case["heads"], device=dev)
    if own:
        import rank_recurrent_state_amd as rrs
        s["cache"] = rrs.Cache(s["k_pages"], s["v_pages"], s["table"])
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import rank_recurrent_state_amd as rrs
        if c["op"] == "rotate":
            rrs.seed_rotate_rows(s["rotary"], s["x"], s["positions"], s["y"])
            return {"y": s["y"]}
        if c["op"] == "verify":
            rrs.seed_verify_drafts(s["target"], s["drafts"], s["uniforms"], s["draws"], s["tokens"], s["counts"], s["offsets"],
                                   draft=s["draft"])
            return {"tokens": s["tokens"], "counts": s["counts"]}
        one = len(s["rows"]) == s["q"].shape[0]  # one new token each: no offsets needed
        offsets = None if one else s["offsets"]
        if c["op"] == "append":
            rrs.seed_cache_append(s["cache"], s["lengths"], s["k"], s["v"], offsets=offsets, rotary=s["rotary"], q=s["q"],
                                  q_out=s["q_out"])
            return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        rrs.seed_decode_attend(s["cache"], s["lengths"], s["q"], s["o"], offsets=offsets, max_tokens=c["fresh"],
                               max_length=max(s["length_list"]), window=c["window"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "rotate":
        return {"y": _turned(s, s["x"], s["positions"])}
    if c["op"] == "verify":
        return _plain_verify(s)
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _turned(s, x, positions):
    c = s["case"]
    angle = 2 * math.pi * torch.frac(positions.double()[:, None] * s["turns"])  # 64 bits: far positions
    cos, sin = (_amplitude(c) * torch.cos(angle)).float()[:, None], (_amplitude(c) * torch.sin(angle)).float()[:, None]
    y, half = x.float().clone(), c["rot"] // 2
    first, second = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else (slice(0, half), slice(half, c["rot"]))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first] = a * cos - b * sin
    y[..., second] = a * sin + b * cos
    return y.to(x.dtype)


def _places(s):
    """Each new row's request and its position in it."""
    starts, n = s["offsets"].long(), sum(s["rows"])
    row = torch.arange(n, device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return seq, s["lengths"].long()[seq] - (starts[seq + 1] - row)


def _plain_append(s):
    page = s["case"]["page"]
    seq, pos = _places(s)
    number = s["table"][seq, pos // page].long()
    s["k_pages"][number, pos % page] = _turned(s, s["k"], pos)
    s["v_pages"][number, pos % page] = s["v"]
    return {"q": _turned(s, s["q"], pos), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    c, q = s["case"], s["q"]
    heads, kh, dim, page = c["heads"], c["key_heads"], c["dim"], c["page"]
    share, fresh = heads // kh, c["fresh"]
    seq, pos = _places(s)
    starts = s["offsets"].long()
    place = torch.arange(len(seq), device=q.device) - starts[seq]
    o = torch.empty(len(seq), heads, dim, device=q.device)
    lse = torch.empty(len(seq), heads, device=q.device)
    lens, b0 = s["length_list"], 0
    while b0 < c["batch"]:  # requests side by side, as many as fit 2 GB of fp32 keys
        b1, longest = b0, 0
        while b1 < c["batch"] and (b1 == b0 or (b1 + 1 - b0) * max(longest, lens[b1]) * kh * dim * 4 <= 2 << 30):
            longest = max(longest, lens[b1])
            b1 += 1
        n, width = b1 - b0, -(-longest // page)
        number = s["table"][b0:b1, :width].long()
        keys, values = (x[number].reshape(n, width * page, kh, dim).permute(0, 2, 1, 3).float() for x in (s["k_pages"], s["v_pages"]))
        here = (seq >= b0) & (seq < b1)
        at, slot = seq[here] - b0, place[here]
        padded = torch.zeros(n, fresh, kh, share, dim, device=q.device)
        where = torch.full((n, fresh), -1, device=q.device)
        padded[at, slot] = q[here].reshape(-1, kh, share, dim).float()
        where[at, slot] = pos[here]
        rows = padded.permute(0, 2, 1, 3, 4).reshape(n, kh, fresh * share, dim)
        scores = torch.matmul(rows, keys.transpose(-1, -2).contiguous()) * dim ** -0.5
        j = torch.arange(width * page, device=q.device)
        seen = j <= where[..., None]
        if c["window"] > 0:
            seen &= j > where[..., None] - c["window"]
        seen = seen.repeat_interleave(share, 1)[:, None]
        scores = torch.where(seen, scores, -torch.inf)
        top = scores.amax(-1, keepdim=True).clamp_min(-3e38)  # padding rows see nothing
        weight = torch.exp(scores - top)
        total = weight.sum(-1, keepdim=True)
        values = torch.where((j < s["lengths"][b0:b1, None])[:, None, :, None], values, 0.0)
        got = (torch.matmul(weight, values) / total).reshape(n, kh, fresh, share, dim).transpose(1, 2)
        logs = (top + torch.log(total)).reshape(n, kh, fresh, share).transpose(1, 2)
        o[here] = got[at, slot].reshape(-1, heads, dim)
        lse[here] = logs[at, slot].reshape(-1, heads)
        b0 = b1
    return {"o": o.to(q.dtype), "lse": lse}


def _plain_verify(s):
    starts = s["offsets"].long()
    rows = starts[1:] - starts[:-1]
    n = len(s["drafts"])
    row = torch.arange(n, device=starts.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    x = s["drafts"].long()[:, None]
    # 64 bits: values next to a border
    p = s["target"].gather(1, x)[:, 0].double()
    q = s["draft"].gather(1, x)[:, 0].double() if s["draft"] is not None else 1.0
    refused = ~(s["uniforms"].double() * q < p) | (row == starts[seq + 1] - 1)  # the last row has no draft
    kept = torch.full_like(rows, n).scatter_reduce(0, seq, torch.where(refused, row, n), "amin") - starts[:-1]
    at = starts[:-1] + kept
    weight, drafted = s["target"][at].double(), kept < rows - 1
    if s["draft"] is not None:
        weight -= torch.where(drafted[:, None], s["draft"][at].double(), 0.0)
    else:
        weight = torch.where(drafted[:, None] & (torch.arange(weight.shape[1], device=x.device) == x[at]), 0.0, weight)
    cum = weight.clamp_min_(0).cumsum(-1)
    last = (weight > 0).long().cumsum(-1).argmax(-1)
    drawn = torch.searchsorted(cum, s["draws"].double()[:, None] * cum[:, -1:], right=True)[:, 0].minimum(last)
    place = row - starts[seq]
    tokens = torch.where(place < kept[seq], s["drafts"], torch.where(place == kept[seq], drawn[seq].to(torch.int32), -1))
    return {"tokens": tokens.to(torch.int32), "counts": (kept + 1).to(torch.int32)}


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "rotate":
        cells = case["rows"] * case["heads"]
        return {"bytes": 2 * cells * case["dim"] * e + 4 * case["rows"], "flops": 3 * cells * case["rot"]}
    rows = _rows_of(case)
    n = sum(rows)
    if op == "verify":
        per = case["vocab"] * e * (2 if case["sampled"] else 1)
        return {"bytes": case["batch"] * per + n * (2 * e + 12), "flops": 3 * case["batch"] * case["vocab"]}
    lens = _lengths(case, rows)
    if op == "append":
        cells = n * (case["heads"] + 2 * case["key_heads"]) * case["dim"]
        return {"bytes": 2 * cells * e + 4 * n, "flops": 3 * n * (case["heads"] + case["key_heads"]) * case["rot"]}
    keys, pairs = 0, 0
    for k, length in zip(rows, lens):
        seen = [min(length - k + i + 1, case["window"] or length) for i in range(k)]
        keys += min(length, (case["window"] + k - 1) if case["window"] else length)
        pairs += sum(seen)
    return {"bytes": (2 * keys * case["key_heads"] + 2 * n * case["heads"]) * case["dim"] * e + 4 * n * case["heads"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---- the definitions, in 64 bits ------------------------------------------------------------------

def _spun(x, positions, case):
    """x [rows, heads, dim] as complex numbers times e^(i angle)."""
    rot = case["rot"]
    t = torch.tensor(_turns(case), dtype=torch.float64, device=x.device)
    angle = positions.double()[:, None] * t
    angle = (angle - torch.round(angle)) * (2 * math.pi)
    turn = torch.polar(torch.full_like(angle, _amplitude(case)), angle)[:, None]
    head = x[..., :rot].double()
    pairs = head.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out = out.flatten(-2) if case["interleaved"] else out.transpose(-1, -2).flatten(-2)
    return torch.cat([out, x[..., rot:].double()], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return {"y": _spun(s["x"], s["positions"], case)}
    ends = [0]
    for k in s["rows"]:
        ends.append(ends[-1] + k)
    if op == "verify":
        tokens, counts = torch.full((ends[-1],), -1, dtype=torch.int32), []
        drafts, uniforms, draws = s["drafts"].tolist(), s["uniforms"].tolist(), s["draws"].tolist()
        for b in range(case["batch"]):
            lo, hi = ends[b], ends[b + 1]
            r = lo
            while r < hi - 1:  # the drafts in turn, until one is refused
                x = drafts[r]
                q = float(s["draft"][r, x]) if case["sampled"] else 1.0
                if not uniforms[r] * q < float(s["target"][r, x]):
                    break
                tokens[r] = x
                r += 1
            w = s["target"][r].double()
            if r < hi - 1 and case["sampled"]:
                w = (w - s["draft"][r].double()).clamp_min(0)
            elif r < hi - 1:
                w[drafts[r]] = 0
            cum = w.cumsum(0)
            hit = (cum > draws[b] * cum[-1]) & (w > 0)
            tokens[r] = int(hit.int().argmax()) if hit.any() else int(torch.nonzero(w > 0)[-1])
            counts.append(r - lo + 1)
        return {"tokens": tokens.cuda(), "counts": torch.tensor(counts, dtype=torch.int32).cuda()}
    page, lens = case["page"], s["length_list"]
    if op == "append":
        pos = torch.cat([torch.arange(n - k, n) for n, k in zip(lens, s["rows"])]).cuda()
        seq = torch.repeat_interleave(torch.arange(case["batch"]), torch.tensor(s["rows"])).cuda()
        number, slot = s["table"][seq, pos // page].long(), pos % page
        keys, values = s["k_pages"].double(), s["v_pages"].double()
        keys[number, slot], values[number, slot] = _spun(s["k"], pos, case), s["v"].double()
        return {"q": _spun(s["q"], pos, case), "k_pages": keys, "v_pages": values}
    heads, kh, dim = case["heads"], case["key_heads"], case["dim"]
    o = torch.empty(ends[-1], heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(ends[-1], heads, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        j = torch.arange(length, device="cuda")
        number, slot = s["table"][b, j // page].long(), j % page
        for h in range(kh):
            K, V = s["k_pages"][number, slot, h].double(), s["v_pages"][number, slot, h].double()
            hs = slice(h * (heads // kh), (h + 1) * (heads // kh))
            for i in range(s["rows"][b]):
                last = length - s["rows"][b] + i
                first = max(0, last + 1 - case["window"]) if case["window"] else 0
                z = (s["q"][ends[b] + i, hs].double() @ K[first:last + 1].T) / math.sqrt(dim)
                lse[ends[b] + i, hs] = torch.logsumexp(z, -1)
                o[ends[b] + i, hs] = torch.softmax(z, -1) @ V[first:last + 1]
    return {"o": o, "lse": lse}
