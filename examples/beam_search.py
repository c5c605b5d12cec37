"""Beam search over a paged cache with one decoder layer, from tokens to tokens, everything on the GPU.

    python examples/beam_search.py [--cache f16|int8|q4_0] [--select PAGES]

A step embeds each beam's token, makes q|k|v by a stacked CBK4 handle, turns q and k to the token's position on their way into
the cache (``KVCache.write_rotated``), attends (``KVCache.attend``, or over the pages that their key summaries select), and gives
the hidden row to a CBK8 head; ``beam_select`` chooses the beams' successors, ``PagePool.fork`` makes their page tables, and
``copy_pages`` copies the pages that they have filled in part.  No number returns to the host before the end: the prompt's pages
are shared by all beams, those of beams that end are given out again, and the cache is packed at the end.  Random weights.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_gb300 import inputs, qgemv  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE, VOCAB = 1024, 8, 2, 128, 16, 4001


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    def __init__(self):
        heads, g = [Q_HEADS, KV_HEADS, KV_HEADS], torch.Generator(device="cuda").manual_seed(1)
        few, many = inputs.cbk_centroids(16), inputs.cbk_centroids(256)
        draw = lambda tag, n, bits, cb: inputs.cbk_packed(inputs.rng("beam_search/" + tag), n, HIDDEN, bits, inputs.cbk_cell_probs(cb))  # noqa: E731
        self.qkv = qgemv.QGemv.stacked("cbk4", [h * DIM for h in heads], HIDDEN, draw("qkv", sum(heads) * DIM, 4, few), None,
                                       np.concatenate([few] * 3))
        self.o = qgemv.QGemv("cbk4", HIDDEN, Q_HEADS * DIM, draw("o", HIDDEN, 4, few), None, few)
        self.head = qgemv.QGemv("cbk8", VOCAB, HIDDEN, draw("head", VOCAB, 8, many), None, many)
        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").half()
        self.rotary = qgemv.Rotary(DIM, [DIM // 2])

    def project(self, tokens):
        """x, and q, k, v [n, heads, DIM] as slices of one product, in calls of at most 16 rows."""
        x = self.embedding[tokens.long()]
        y = torch.cat([self.qkv.gemv(part) for part in x.split(16)]).unflatten(1, (-1, DIM))
        return x, y[:, :Q_HEADS], y[:, Q_HEADS:Q_HEADS + KV_HEADS], y[:, Q_HEADS + KV_HEADS:]

    def logits(self, x, attended):
        h = torch.cat([self.o.run_residual(a.flatten(1).contiguous(), torch.empty_like(r), r)
                       for a, r in zip(attended.split(16), x.float().split(16))])
        return torch.cat([self.head.gemv((part / 8).half()) for part in h.split(16)])


class Search:
    """`beams` continuations of one prompt."""

    def __init__(self, model, prompt, beams, steps, cache="int8", select=0, pages=200):
        self.model, self.beams, self.select = model, beams, select
        self.cache = qgemv.KVCache(cache, pages, PAGE, KV_HEADS, DIM)
        self.pool = qgemv.PagePool(pages, PAGE)
        self.summary = qgemv.KeySummary(self.cache)
        self.ws = qgemv.AttnWorkspace(beams, Q_HEADS, DIM)
        self.beam_ws = qgemv.BeamWorkspace(1, beams, VOCAB, beams)
        entries = -(-(len(prompt) + steps) // PAGE)
        self.length = len(prompt) - 1  # cached tokens of each beam
        # the prompt but for its last token, once; then a row for each beam
        table = torch.full((1, entries), -1, dtype=torch.int32, device="cuda")
        self.pool.reserve(table, ints(0), ints(self.length))
        _, q, k, v = model.project(prompt[:-1])
        at = torch.arange(self.length, device="cuda")
        self.cache.write_rotated(model.rotary, q, k, v, at[:, None].int(), table[0, at // PAGE].long() * PAGE + at % PAGE)
        self.summary.update(table[0, :self.length // PAGE].contiguous())
        self.table = self.fork(table, torch.zeros(beams, dtype=torch.int32, device="cuda"), ints(self.length))
        self.tokens = prompt[-1:].repeat(beams)
        self.history = torch.empty(beams, 0, dtype=torch.int32, device="cuda")
        # all beams are the same at first: one of them is in use
        self.scores = torch.full((1, beams), -float("inf"), device="cuda")
        self.scores[0, 0] = 0

    def fork(self, table, parents, lens):
        table, src, dst, tokens = self.pool.fork(table, parents, lens)
        self.cache.copy_pages(src, dst, tokens)
        return table

    def step(self):
        n, at, dev = self.beams, self.length, "cuda"
        lens = torch.full((n,), at, dtype=torch.int32, device=dev)
        self.pool.reserve(self.table, lens, lens + 1)
        x, q, k, v = self.model.project(self.tokens)
        slots = self.table[:, at // PAGE].long() * PAGE + at % PAGE
        q = self.cache.write_rotated(self.model.rotary, q, k, v, lens[:, None], slots)
        cu = torch.arange(n + 1, dtype=torch.int32, device=dev)
        if self.select:
            pages, ctx = self.cache.select(q, self.table, lens, cu, summary=self.summary, n_select=self.select)
            out, _ = self.cache.attend_pages(q, pages, ctx, cu, max_ctx=(self.select + 1) * PAGE, max_new=1, workspace=self.ws)
        else:
            out, _ = self.cache.attend(q, self.table, lens, cu, max_ctx=at, max_new=1, workspace=self.ws)
        self.length += 1
        if self.length % PAGE == 0:  # the beams' last pages have become full
            self.summary.update(self.table[:, at // PAGE].contiguous())
        scores, parents, tokens = qgemv.beam_select(self.model.logits(x, out), self.scores, n, workspace=self.beam_ws)
        self.table = self.fork(self.table, parents[0], lens + 1)
        self.scores, self.tokens = scores, tokens[0]
        self.history = torch.cat([self.history[parents[0].long()], self.tokens[:, None]], 1)

    def pack(self):
        self.table, src, dst = self.pool.compact(self.table)
        self.cache.copy_pages(src, dst)
        self.summary.update(dst)  # what lies there now


def run(cache="int8", beams=5, steps=40, prompt=100, select=0):
    """(the search when it has ended, its prompt)."""
    tokens = torch.randint(0, VOCAB, (prompt,), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    search = Search(Model(), tokens, beams, steps, cache, select)
    for _ in range(steps):
        search.step()
    search.pack()
    search.pool.status()
    search.ws.status()
    return search, tokens


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=sorted(qgemv.KV_FORMATS), default="int8")
    ap.add_argument("--select", type=int, default=0, help="pages that a token attends besides the last ones (0: all)")
    a = ap.parse_args()
    got, _ = run(a.cache, select=a.select)
    print(f"{got.history.shape[1]} tokens of {got.beams} beams: scores {got.scores[0].tolist()}, {int((got.pool.refs > 0).sum())} pages in use")
