"""The example's beam search against a plain decoder in 64 bits: the same dequantised weights,
no cache, no pages, every hypothesis recomputed from its tokens.

Tolerance. q, k, v and the attention's output are rounded to f16 (2^-11 each) between products
that keep their inputs' size, in 2 layers; logits have a size of about 2, so a log
probability moves by some 2 * 2 * 4 * 2^-11 = 0.008 at most, and a score by that for each of its tokens.
"""
import os
import sys

import pytest
import torch

import bit_ternary_matmul_gb300 as q

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

PER_TOKEN = 0.008


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    q.build()
    import beam_decode
    return beam_decode


class Plain:
    def __init__(self, m):
        def dense(w, n, k):
            return q.q2_0_get_rows(w, n, k, torch.arange(n, dtype=torch.int32, device="cuda")).double()
        self.m = m
        self.embed = dense(m.embed, m.vocab, m.hidden)
        self.head = dense(m.head, m.vocab, m.hidden)
        nq = (m.n_q + 2 * m.n_kv) * m.dim
        self.blocks = [dict(qkv=dense(b["qkv"], nq, m.hidden), o=dense(b["o"], m.hidden, m.n_q * m.dim),
                            up=dense(b["up"], 2 * m.inner, m.hidden), down=dense(b["down"], m.hidden, m.inner))
                       for b in m.blocks]

    def log_probs(self, tokens):
        """[len][vocab] of one sequence."""
        m, t = self.m, len(tokens)
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        x = self.embed[torch.tensor(tokens, device="cuda")]
        h = m.dim // 2
        c, s = m.rope[:t, None, :h].double(), m.rope[:t, None, h:].double()
        turn = lambda y: torch.cat([y[..., :h] * c - y[..., h:] * s, y[..., :h] * s + y[..., h:] * c], -1)  # noqa: E731
        mask = torch.ones((t, t), dtype=torch.bool, device="cuda").tril()
        for b in self.blocks:
            qkv = (norm(x) @ b["qkv"].T).reshape(t, -1, m.dim)
            qq, k, v = turn(qkv[:, : m.n_q]), turn(qkv[:, m.n_q: m.n_q + m.n_kv]), qkv[:, m.n_q + m.n_kv:]
            k, v = (y.repeat_interleave(m.n_q // m.n_kv, 1) for y in (k, v))
            p = torch.einsum("ihd,jhd->hij", qq, k) * m.dim ** -0.5
            p = torch.softmax(p.masked_fill(~mask, float("-inf")), -1)
            x = x + torch.einsum("hij,jhd->ihd", p, v).reshape(t, -1) @ b["o"].T
            gate, up = (norm(x) @ b["up"].T).split(m.inner, 1)
            x = x + (torch.nn.functional.silu(gate) * up) @ b["down"].T
        return torch.log_softmax(norm(x) @ self.head.T, -1)

    def beam_search(self, prompt, beams, steps):
        hyps = [((), 0.0)]
        for _ in range(steps + 1):
            cands = []
            for h, s in hyps:
                lp = self.log_probs(list(prompt) + list(h))[-1] + s
                top = torch.topk(lp, beams)
                cands += [(h + (int(i),), float(v)) for v, i in zip(top.values, top.indices)]
            hyps = sorted(cands, key=lambda c: -c[1])[:beams]
        return hyps


@pytest.mark.parametrize("beams,prompt_len,steps,kw", [
    (4, 37, 20, {}), (1, 5, 18, {}), (8, 130, 35, {}), (3, 16, 17, dict(n_kv=8, page=32)),
    (5, 50, 10, dict(n_q=4, n_kv=1, dim=128, dtype=torch.bfloat16))])
def test_beam_decode_against_plain(example, beams, prompt_len, steps, kw):
    model = example.Decoder(seed=beams, **kw)
    g = torch.Generator().manual_seed(prompt_len)
    prompt = torch.randint(0, model.vocab, (prompt_len,), generator=g).tolist()
    pages = len(model.free)
    hyps, scores = example.beam_search(model, prompt, beams, steps)
    assert len(hyps) == beams and all(len(h) == steps + 1 for h in hyps)
    assert scores == sorted(scores, reverse=True) and len({tuple(h) for h in hyps}) == beams
    # what is not free: the prompt's pages and at most each beam's own
    assert pages - len(model.free) <= -(-prompt_len // model.page) + beams * (steps // model.page + 1)
    plain = Plain(model)
    tol = PER_TOKEN * (steps + 1) * (8 if kw.get("dtype") == torch.bfloat16 else 1)
    for h, s in zip(hyps, scores):
        lp = plain.log_probs(prompt + h)
        e = sum(float(lp[len(prompt) - 1 + i, t]) for i, t in enumerate(h))
        assert abs(s - e) <= tol, (s, e)
    if beams * steps <= 100:
        best = plain.beam_search(prompt, beams, steps)[0][1]
        assert abs(best - scores[0]) <= tol


def test_beams_stop_at_the_end_token(example):
    model = example.Decoder(seed=3)
    hyps, scores = example.beam_search(model, [1, 2, 3], 4, 6)
    end = hyps[0][2]
    hyps, scores = example.beam_search(example.Decoder(seed=3), [1, 2, 3], 4, 12, end=end)
    for h in hyps:
        if end in h:
            assert all(t == end for t in h[h.index(end):])


@pytest.mark.parametrize("at", [0, 2, 4])
def test_a_finished_beam_keeps_its_score(example, at):
    """With an end token that the best hypothesis contains, that hypothesis is finished there and only loses
    to better ones: some hypothesis ends, and the score of each that does is that of its tokens up to the end."""
    prompt = [1, 2, 3]
    end = example.beam_search(example.Decoder(seed=3), prompt, 4, 6)[0][0][at]
    model = example.Decoder(seed=3)
    hyps, scores = example.beam_search(model, prompt, 4, 12, end=end)
    assert any(end in h for h in hyps), "no hypothesis ended"
    assert scores == sorted(scores, reverse=True) and len({tuple(h) for h in hyps}) == 4
    plain = Plain(model)
    for h, s in zip(hyps, scores):
        n = h.index(end) + 1 if end in h else len(h)
        assert all(t == end for t in h[n:])
        lp = plain.log_probs(prompt + h[:n])
        e = sum(float(lp[len(prompt) - 1 + i, t]) for i, t in enumerate(h[:n]))
        assert abs(s - e) <= PER_TOKEN * n, (s, e)
