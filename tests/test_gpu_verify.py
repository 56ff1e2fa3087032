"""GPU tests of draft verification (seed_verify_drafts) against the plain fp64 form of attend_ref.py.
Results are whole numbers and equal; the sums' order moves a border between tokens by at most 1e-13, so draws
that are meant to meet a border are dyadic fractions, whose sums are exact in any order."""
from __future__ import annotations

import numpy as np
import pytest

import attend_ref as ref

pytestmark = pytest.mark.gpu


def _rrs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_recurrent_state_amd as rrs
    return rrs, torch


def _run(rrs, torch, target, draft, drafts, uniforms, draws, offsets, **kw):
    """Arrays or tensors in; checks out and counts against the definition."""
    def dev(x, dt):
        return None if x is None else x if torch.is_tensor(x) else torch.tensor(np.asarray(x), dtype=dt, device="cuda")

    target, draft = dev(target, torch.float32), dev(draft, torch.float32)
    drafts, offsets = dev(drafts, torch.int32), dev(offsets, torch.int32)
    uniforms, draws = dev(uniforms, torch.float32), dev(draws, torch.float32)
    out = torch.full_like(drafts, -2)
    counts = torch.full((len(offsets) - 1,), -3, dtype=torch.int32, device="cuda")
    rrs.seed_verify_drafts(target, drafts, uniforms, draws, out, counts, offsets, draft=draft, **kw)
    torch.cuda.synchronize()

    def host(x):
        return None if x is None else x.double().cpu().numpy()

    wo, wc = ref.verify(host(target), host(draft), drafts.cpu().numpy(), host(uniforms), host(draws), offsets.cpu().numpy())
    assert np.array_equal(out.cpu().numpy(), wo) and np.array_equal(counts.cpu().numpy(), wc)
    return out, counts


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 63, 1000, 4096, 4097, 100003])
def test_random(dtype, sampled, vocab):
    rrs, torch = _rrs()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows = [1, 5, 0, 9, 2, 70 if vocab < 5000 else 4, 1, 0, 3]
    n = sum(rows)
    logits = 2 * torch.randn(n, vocab, generator=g, device="cuda")
    target = torch.softmax(logits, -1).to(dt)
    near = logits + 0.4 * torch.randn(n, vocab, generator=g, device="cuda")
    draft = torch.softmax(near, -1).to(dt)
    drafts = torch.multinomial(draft.float(), 1, generator=g)[:, 0].to(torch.int32) if sampled else near.argmax(-1).to(torch.int32)
    offsets = np.concatenate([[0], np.cumsum(rows)])
    for i in range(3):
        u = torch.rand(n, generator=g, device="cuda") * (1.0 if i else 0.05)  # mostly kept, then as they come
        r = torch.rand(len(rows), generator=g, device="cuda")
        _run(rrs, torch, target, draft if sampled else None, drafts, u, r, offsets)


def test_borders():
    """Draws on and next to the borders between tokens, exact in any order of summing."""
    rrs, torch = _rrs()
    vocab = 8192
    p = np.zeros((1, vocab), np.float32)
    p[0, ::2] = 1.0 / 4096
    for k in (0, 1, 2, 2047, 2048, 2049, 4095):
        for shift, token in ((0.0, 2 * k), (-2.0 ** -26, 2 * k - 2), (2.0 ** -26, 2 * k)):
            r = k / 4096 + shift
            if r < 0:
                continue
            out, _ = _run(rrs, torch, p, None, [0], [0.5], [np.float32(r)], [0, 1])
            if float(np.float32(r)) == r:  # the shift is not lost in rounding
                assert int(out[0]) == token, (k, shift)


def test_acceptance_border():
    """u q < p, exactly: equality refuses."""
    rrs, torch = _rrs()
    p = np.tile(np.float32([0.25, 0.75]), (2, 1))
    q = np.tile(np.float32([0.5, 0.5]), (2, 1))
    out, counts = _run(rrs, torch, p, q, [0, 0], [0.5, 0.0], [0.3], [0, 2])
    assert int(counts[0]) == 1 and int(out[0]) == 1
    out, counts = _run(rrs, torch, p, q, [0, 0], [np.nextafter(np.float32(0.5), np.float32(0)), 0.0], [0.3], [0, 2])
    assert int(counts[0]) == 2 and out.tolist() == [0, 1]


def test_degenerate_rows():
    """Weights of zero, negative, NaN and infinite; drafts that are no tokens; draws of 1."""
    rrs, torch = _rrs()
    nan, inf = float("nan"), float("inf")
    vocab = 5000
    rng = np.random.default_rng(1)
    base = rng.random(vocab).astype(np.float32)
    base /= base.sum()
    zero = np.zeros(vocab, np.float32)
    for row in (zero, np.full(vocab, nan, np.float32), -base, np.where(np.arange(vocab) == 4321, 1, 0).astype(np.float32),
                np.where(np.arange(vocab) % 7 == 0, nan, base).astype(np.float32)):
        for r in (0.0, 0.5, 1.0, 2.0, nan):
            _run(rrs, torch, row[None], None, [3], [0.5], [r], [0, 1])
    # refused with nothing left of p - q: the draw is from p
    for x in (-1, vocab, 1 << 30, -(1 << 31), 17):
        p = np.stack([base, base])
        q = p.copy()
        p[:, 17] = q[:, 17] = 0
        out, counts = _run(rrs, torch, p, q, [x, 0], [0.5, 0.5], [0.7], [0, 2])
        assert int(counts[0]) == 1 and 0 <= int(out[0]) < vocab and int(out[1]) == -1
        _run(rrs, torch, p, None, [x, 0], [0.5, 0.5], [0.7], [0, 2])
    # infinite weights: no running sum passes, the last token of positive weight is taken
    row = base.copy()
    row[100] = inf
    out = torch.empty(1, dtype=torch.int32, device="cuda")
    counts = torch.empty_like(out)
    t = torch.tensor(row[None], device="cuda")
    one = torch.ones(1, device="cuda")
    rrs.seed_verify_drafts(t, out.zero_().clone(), one, 0.5 * one, out, counts, torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert int(out[0]) == vocab - 1 and int(counts[0]) == 1


def test_rows_in_place_and_strided():
    """out may be drafts; rows of wider buffers at any alignment; rows of no request stay as they are."""
    rrs, torch = _rrs()
    g = torch.Generator(device="cuda").manual_seed(2)
    vocab, n = 4501, 12
    for dt in (torch.float32, torch.bfloat16):
        for shift in (0, 1, 5):
            wide = torch.rand(n, vocab + 9, generator=g, device="cuda").to(dt)
            other = torch.rand(n, vocab + 20, generator=g, device="cuda").to(dt)
            p, q = wide[:, shift:shift + vocab], other[:, 3:3 + vocab]
            drafts = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
            u, r = torch.rand(n, generator=g, device="cuda"), torch.rand(3, generator=g, device="cuda")
            offsets = torch.tensor([2, 5, 5, 10], dtype=torch.int32, device="cuda")
            out, counts = _run(rrs, torch, p, q, drafts, u, r, offsets)
            same, c2 = drafts.clone(), torch.empty_like(counts)
            ws = torch.full((rrs.seed_verify_workspace_bytes(3, vocab),), 255, dtype=torch.uint8, device="cuda")
            rrs.seed_verify_drafts(p, same, u, r, same, c2, offsets, draft=q, ws=ws)
            assert torch.equal(torch.where(out == -2, drafts, out), same) and torch.equal(counts, c2)
    # wrong offsets stay inside the buffers
    for offsets in ([5, 1, 100, 3], [-4, 30, 2, 12], [1 << 30, -(1 << 31), 0, 12]):
        out = torch.full_like(drafts, -2)
        rrs.seed_verify_drafts(p, drafts, u, r, out, counts, torch.tensor(offsets, dtype=torch.int32, device="cuda"), draft=q)
        torch.cuda.synchronize()
        assert int(out.max()) < vocab


def test_graph_replays():
    rrs, torch = _rrs()
    g = torch.Generator(device="cuda").manual_seed(3)
    vocab, n = 20000, 9
    offsets = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    p, q = torch.empty(n, vocab, device="cuda"), torch.empty(n, vocab, device="cuda")
    drafts, u, r = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    out, counts = torch.empty_like(drafts), torch.empty(2, dtype=torch.int32, device="cuda")

    def fill():
        z = 2 * torch.randn(n, vocab, generator=g, device="cuda")
        p.copy_(torch.softmax(z, -1))
        q.copy_(torch.softmax(z + 0.3 * torch.randn(n, vocab, generator=g, device="cuda"), -1))
        drafts.copy_(torch.multinomial(q, 1, generator=g)[:, 0])
        u.uniform_(generator=g)
        r.uniform_(generator=g)

    fill()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        rrs.seed_verify_drafts(p, drafts, u, r, out, counts, offsets, draft=q)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        rrs.seed_verify_drafts(p, drafts, u, r, out, counts, offsets, draft=q)
    for _ in range(5):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        wo, wc = _run(rrs, torch, p, q, drafts, u, r, offsets)
        assert torch.equal(out, wo) and torch.equal(counts, wc)
