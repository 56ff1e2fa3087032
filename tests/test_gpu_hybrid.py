"""A small hybrid model served with the library: a recurrent (Gated DeltaNet) layer and an attention layer, prompts,
drafted tokens and their verification, against the same model in fp64 that recomputes every sequence from its
tokens. Tokens are equal: the probabilities differ by rounding (fp32, a few hundred operations: below 1e-4 of each, as
asserted), and no draw of this seed lies that close to a border."""
from __future__ import annotations

import numpy as np
import pytest

import attend_ref as ref
import prompt_ref

pytestmark = pytest.mark.gpu

D, HEADS, KEY_HEADS, VOCAB, PAGE, MOST = 64, 4, 2, 97, 16, 5  # width of a head and of the model, heads, drafts and the token before


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


class Model:
    def __init__(self, seed):
        r = np.random.default_rng(seed)

        def w(*shape):
            return (r.standard_normal(shape) / np.sqrt(shape[0])).astype(np.float32).astype(np.float64)

        self.embed = w(VOCAB, D) * 8
        self.recurrent = {n: w(D, k) for n, k in (("q", 2 * D), ("k", 2 * D), ("v", 2 * D), ("beta", 2), ("g", 2), ("o", 2 * D))}
        self.recurrent["o"] = w(2 * D, D)
        self.attention = {"q": w(D, HEADS * D), "k": w(D, KEY_HEADS * D), "v": w(D, KEY_HEADS * D), "o": w(HEADS * D, D)}
        self.head = w(D, VOCAB) * 2
        self.turns = ref.turns(32, base=500.0)

    def probabilities(self, tokens):
        """fp64, of the token behind every one of `tokens`, with no state kept."""
        h = self.embed[tokens]
        n = len(tokens)
        p = self.recurrent
        q, k, v = ((h @ p[x]).reshape(n, 2, D) for x in "qkv")
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True)) for x in (q, k))
        beta, g = 1 / (1 + np.exp(-h @ p["beta"])), 0.8 + 0.2 / (1 + np.exp(-h @ p["g"]))
        o = prompt_ref.scan(prompt_ref.GDN, [n], q, k, v, beta, g, None)[0]
        h = h + o.reshape(n, 2 * D) @ p["o"]
        p, pos = self.attention, np.arange(n)
        q, k, v = (h @ p["q"]).reshape(n, HEADS, D), (h @ p["k"]).reshape(n, KEY_HEADS, D), (h @ p["v"]).reshape(n, KEY_HEADS, D)
        q, k = ref.rotate(q, pos, self.turns)[0], ref.rotate(k, pos, self.turns)[0]
        o = np.stack([ref.attend(q[:, i], k[:, i * KEY_HEADS // HEADS], v[:, i * KEY_HEADS // HEADS], pos, D ** -0.5)[0] for i in range(HEADS)], 1)
        h = h + o.reshape(n, HEADS * D) @ p["o"]
        return _softmax(h @ self.head)


class Served:
    """The model on the GPU: a dense recurrent state and a paged cache per request."""

    def __init__(self, rrs, torch, model, batch, longest):
        self.rrs, self.torch = rrs, torch

        def dev(x):
            return torch.tensor(x, dtype=torch.float32, device="cuda")

        self.embed, self.head = dev(model.embed), dev(model.head)
        self.recurrent = {k: dev(x) for k, x in model.recurrent.items()}
        self.attention = {k: dev(x) for k, x in model.attention.items()}
        self.rotary = rrs.make_rotary(32, base=500.0)
        width = -(-longest // PAGE)
        pool = torch.full((2, batch * width, PAGE, KEY_HEADS, D), float("nan"), device="cuda")  # what was never stored is never seen
        table = torch.randperm(batch * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(batch, width).cuda()
        self.cache = rrs.Cache(pool[0], pool[1], table)
        self.shape = rrs.make_shape(rrs.SEED_GDN, batch, 2, D, D, 16, 16, rrs.SEED_F32)
        self.state = torch.zeros(batch, 2, D, D, device="cuda")
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def rows(self, tokens, offsets, counts):
        """Probabilities behind every new token; the cache takes them all."""
        rrs, torch, n = self.rrs, self.torch, len(tokens)
        self.lengths += counts
        h = self.embed[tokens.long()]
        p = self.recurrent
        q, k, v = ((h @ p[x]).view(n, 2, D) for x in "qkv")
        unit = torch.full((2, D), D ** -0.5, device="cuda")
        for x in (q, k):
            rrs.seed_norm_rows(x, unit, x, eps=0.0)
        beta, g = torch.sigmoid(h @ p["beta"]), 0.8 + 0.2 * torch.sigmoid(h @ p["g"])
        o, after = torch.empty_like(v), torch.empty_like(self.state)
        rrs.seed_prefill_scan(self.shape, offsets, q, k, v, beta, g, after, o, S0=self.state)
        self.last = (q, k, v, beta, g, offsets)
        h = h + o.view(n, 2 * D) @ p["o"]
        p = self.attention
        q, k, v = (h @ p["q"]).view(n, HEADS, D), (h @ p["k"]).view(n, KEY_HEADS, D), (h @ p["v"]).view(n, KEY_HEADS, D)
        rrs.seed_cache_append(self.cache, self.lengths, k, v, offsets=offsets, rotary=self.rotary, q=q, q_out=q)
        o = torch.empty_like(q)
        rrs.seed_decode_attend(self.cache, self.lengths, q, o, offsets=offsets, max_tokens=32)
        return torch.softmax((h + o.view(n, HEADS * D) @ p["o"]) @ self.head, -1)

    def keep(self, kept, given):
        """The first kept[b] of a request's given[b] rows count: the cache by its length, the state by running
        over them again, the others as tokens that change nothing."""
        q, k, v, beta, g, offsets = self.last
        row = self.torch.arange(len(q), device="cuda")
        seq = self.torch.searchsorted(offsets[1:].long(), row, right=True)
        drop = (row - offsets[seq].long() >= kept[seq])[:, None]
        beta, g = self.torch.where(drop, 0.0, beta), self.torch.where(drop, 1.0, g)
        self.rrs.seed_prefill_scan(self.shape, offsets, q, k, v, beta, g, self.state, self.torch.empty_like(v), S0=self.state)
        self.lengths += kept - given


def test_drafted_generation_of_a_hybrid_model():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_recurrent_state_amd as rrs
    r = np.random.default_rng(11)
    model = Model(2)
    prompts = [r.integers(0, VOCAB, n).tolist() for n in (17, 1, 30)]
    served = Served(rrs, torch, model, 3, 128)

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def f32(x):
        return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")

    # the prompts but for their last token, which the first round takes
    counts = [len(p) - 1 for p in prompts]
    given = i32(counts)
    served.rows(i32(sum((p[:-1] for p in prompts), [])), i32(np.concatenate([[0], np.cumsum(counts)])), given)
    served.keep(given, given)
    assert served.lengths.tolist() == counts
    sequences, kept_drafts = [list(p) for p in prompts], 0
    for turn in range(8):
        rows = [int(r.integers(1, MOST + 1)) for _ in prompts]
        ends = np.concatenate([[0], np.cumsum(rows)])
        want_p, tokens, drafts = [], [], []
        draft = np.zeros((ends[-1], VOCAB), np.float32)
        for b, seq in enumerate(sequences):
            line = list(seq)
            for i in range(rows[b] - 1):  # drafts from a blunter copy of the model
                q = _softmax(0.7 * np.log(model.probabilities(np.array(line))[-1])).astype(np.float32)
                draft[ends[b] + i] = q
                line.append(int(r.choice(VOCAB, p=q.astype(np.float64) / q.astype(np.float64).sum())))
            want_p.append(model.probabilities(np.array(line))[len(seq) - 1:])
            tokens += line[len(seq) - 1:]
            drafts += line[len(seq):] + [0]
        want_p = np.concatenate(want_p)
        u, d = r.random(ends[-1]).astype(np.float32), r.random(3).astype(np.float32)
        want, want_counts = ref.verify(want_p, draft.astype(np.float64), np.array(drafts), u.astype(np.float64), d.astype(np.float64), ends)
        given = i32(rows)
        p = served.rows(i32(tokens), i32(ends), given)
        assert (np.abs(p.double().cpu().numpy() - want_p) <= 1e-4 * want_p + 1e-7).all()
        out, counts = i32(drafts), torch.empty(3, dtype=torch.int32, device="cuda")
        rrs.seed_verify_drafts(p, out, f32(u), f32(d), out, counts, i32(ends), draft=f32(draft))
        assert out.tolist() == want.tolist() and counts.tolist() == want_counts.tolist()
        served.keep(counts, given)
        for b in range(3):
            sequences[b] += want[ends[b]:ends[b] + want_counts[b]].tolist()
        kept_drafts += int((want_counts - 1).sum())
        assert served.lengths.tolist() == [len(s) - 1 for s in sequences]
    assert kept_drafts > 8  # some rounds kept some drafts
