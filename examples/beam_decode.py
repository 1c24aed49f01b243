"""Beam search on a small ternary decoder with random weights: the library's calls of a
decode step, together as they would be used.

A prompt goes through the layers at once (grouped products, keys and values appended to the
cache, causal attention as one sequence per token on the same pages). Its pages are then the
shared prefix of the beams. A step takes one token per beam: gathered embeddings, the
projections (decode mat-vec, one column per beam), rotated keys and values appended, attention
over the prefix and each beam's own pages, the head's logits, the selection, and the page
tables reordered after it. PyTorch does the norms, the activation and the additions.

    python examples/beam_decode.py --beams 4 --steps 40
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_ternary_matmul_gb300 as q  # noqa: E402


class Decoder:
    """Weights and cache of a small decoder."""

    def __init__(self, layers=2, hidden=512, n_q=8, n_kv=4, dim=64, inner=1024, vocab=4096, page=16, n_pages=256,
                 max_pos=2048, dtype=torch.float16, seed=0):
        self.layers, self.hidden, self.n_q, self.n_kv, self.dim = layers, hidden, n_q, n_kv, dim
        self.inner, self.vocab, self.page = inner, vocab, page
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(n, k, gain=1.0):
            # ternary weights whose products keep their input's size
            return q.q2_0_quantize_ref(torch.randn((n, k), generator=g, device="cuda") * (gain / k ** 0.5) * 0.5, n, k)

        self.embed = matrix(vocab, hidden, 30.0)
        self.blocks = [dict(qkv=matrix((n_q + 2 * n_kv) * dim, hidden), o=matrix(hidden, n_q * dim),
                            up=matrix(2 * inner, hidden), down=matrix(hidden, inner)) for _ in range(layers)]
        self.head = matrix(vocab, hidden, 3.0)
        shape = (layers, n_pages, n_kv, page, dim)
        self.cache = q.KvCache(torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda"))
        self.free = list(range(n_pages))
        angle = torch.arange(max_pos, device="cuda")[:, None] * 1e4 ** (-torch.arange(0, dim, 2, device="cuda") / dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def product(self, w, x, n):
        """x [tokens][k] times a packed n x k matrix: mat-vec for up to 8 tokens, GEMM above."""
        x = x.contiguous()
        k = x.shape[1]
        if x.dtype == torch.float16:
            return q.q2_0_mul_mat_vec_f16(w, x, n, k) if x.shape[0] <= 8 else q.q2_0_mul_mat_f16(w, x, n, k)
        return q.q2_0_mul_mat_vec(w, x, n, k) if x.shape[0] <= 8 else q.q2_0_mul_mat(w, x, n, k)

    def forward(self, tokens, pos, slot, table, seq, q_buf, plan):
        """Logits [tokens][vocab] of one token per row; keys and values go to (seq, slot) of the table."""
        x = q.q2_0_get_rows(self.embed, self.vocab, self.hidden, tokens)
        n = x.shape[0]
        a, b = self.n_q * self.dim, (self.n_q + self.n_kv) * self.dim
        for i, w in enumerate(self.blocks):
            qkv = self.product(w["qkv"], self.norm(x), b + self.n_kv * self.dim)
            q.q2_0_kv_append(self.cache, i, qkv[:, :a], qkv[:, a:b], qkv[:, b:], pos, slot, table, self.rope, seq=seq,
                             q_out=q_buf)
            att = plan.execute(i).reshape(n, a)
            x = x + self.product(w["o"], att if att.dtype == torch.float16 else att.float(), self.hidden)
            gate, up = self.product(w["up"], self.norm(x), 2 * self.inner).split(self.inner, 1)
            x = x + self.product(w["down"], torch.nn.functional.silu(gate) * up, self.hidden)
        return self.product(self.head, self.norm(x), self.vocab)

    def take(self, n):
        pages, self.free = self.free[:n], self.free[n:]
        return pages


def beam_search(model: Decoder, prompt, beams=4, steps=20, end=None):
    """(tokens [beams][<= steps + 1] lists, scores [beams]) of the best continuations of a prompt."""
    dev = model.embed.device
    i32 = dict(dtype=torch.int32, device=dev)
    dtype, t = model.cache.k.dtype, len(prompt)
    shape = (model.n_q, model.dim)
    # ---- the prompt: token i attends to the first i + 1 tokens of one row of pages
    pages = model.take(-(-t // model.page))
    prefix = torch.tensor([pages], **i32)
    place = torch.arange(t, **i32)
    q_buf, out = (torch.empty((t, *shape), dtype=dtype, device=dev) for _ in range(2))
    rows = prefix.expand(t, -1).contiguous()
    plan = q.AttnPlan(model.cache, q_buf, out, rows, place + 1)
    logits = model.forward(torch.tensor(prompt, **i32), place, place, prefix, torch.zeros(t, **i32), q_buf, plan)
    torch.cuda.synchronize()
    plan.close()
    score, parent, token = q.q2_0_beam_select(logits[-1].reshape(1, 1, -1), torch.zeros((1, 1), device=dev), beams)
    hyps = [[x] for x in token[0].tolist()]
    # ---- the beams: own pages behind the shared ones
    width = -(-steps // model.page) + 1
    table = torch.full((beams, width), -1, **i32)
    table[:, 0] = torch.tensor(model.take(beams), **i32)
    length = torch.zeros(beams, **i32)      # tokens in the cache, and with the one being added
    with_new = torch.ones(beams, **i32)
    q_buf, out = (torch.empty((beams, *shape), dtype=dtype, device=dev) for _ in range(2))
    plan = q.AttnPlan(model.cache, q_buf, out, table, with_new, prefix, torch.tensor([t], **i32))
    done = torch.zeros((1, beams), dtype=torch.uint8, device=dev)
    for _ in range(steps):
        logits = model.forward(token[0].clamp(min=0), length + t, length, table, None, q_buf, plan)
        if end is not None:  # a beam is finished from its end token on
            done = torch.gather(done, 1, parent.long()) | (token == end).to(torch.uint8)
        score, parent, token = q.q2_0_beam_select(logits.reshape(1, beams, -1), score, beams, done=done,
                                                  done_token=-1 if end is None else end)
        # ---- the tables follow; pages that no row names any more are free again
        fresh = model.take(beams)
        new_table, new_length, used = q.q2_0_beam_reorder(model.cache, parent, table, with_new, torch.tensor(fresh, **i32))
        held = {p for r in table.tolist() for p in r if p >= 0} | set(fresh)
        table.copy_(new_table)
        length.copy_(new_length)
        with_new.copy_(new_length + 1)
        live = {p for r, n in zip(table.tolist(), length.tolist()) for p in r[: n // model.page + 1]}
        model.free += sorted(held - live)
        hyps = [hyps[p] + [x] for p, x in zip(parent[0].tolist(), token[0].tolist())]
    torch.cuda.synchronize()
    plan.close()
    code, info = q.q2_0_get_error()
    if code:
        raise RuntimeError(f"device error {code} ({info})")
    return hyps, score[0].tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prompt", type=int, default=100, help="length of the random prompt")
    a = ap.parse_args()
    q.build()
    model = Decoder()
    g = torch.Generator().manual_seed(1)
    hyps, scores = beam_search(model, torch.randint(0, model.vocab, (a.prompt,), generator=g).tolist(), a.beams, a.steps)
    for h, s in zip(hyps, scores):
        print("%9.4f  %s" % (s, " ".join(map(str, h))))


if __name__ == "__main__":
    main()
