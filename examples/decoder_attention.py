"""The attention of one decoder layer, from packed projections to the o product: a prompt in two chunks, then drafted
tokens that are verified together, and the accepted ones kept.

    python examples/decoder_attention.py [--cache f16|int8|q4_0]

Everything runs on the GPU through the library: q|k|v by one stacked CBK4 handle (at most 16 rows a call), the cache by
``KVCache``, the prompt by ``attn_prompt``, the drafts by ``KVCache.attend``, o and the residual by another handle.  Random
weights; no positions are encoded (a model would rotate q and k between the projection and the cache).  The drafts' outputs are
compared with the same tokens' as a prompt.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_gb300 import inputs, qgemv  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, PAGE = 1024, 8, 2, 128, 16


class Layer:
    def __init__(self, cache, pages=64):
        heads = [Q_HEADS, KV_HEADS, KV_HEADS]
        cb = inputs.cbk_centroids(16)
        draw = lambda tag, n, k: inputs.cbk_packed(inputs.rng("decoder_attention/" + tag), n, k, 4, inputs.cbk_cell_probs(cb))  # noqa: E731
        import numpy as np
        self.qkv = qgemv.QGemv.stacked("cbk4", [h * DIM for h in heads], HIDDEN, draw("qkv", sum(heads) * DIM, HIDDEN),
                                       None, np.concatenate([cb] * 3))
        self.o = qgemv.QGemv("cbk4", HIDDEN, Q_HEADS * DIM, draw("o", HIDDEN, Q_HEADS * DIM), None, cb)
        self.cache = qgemv.KVCache(cache, pages, PAGE, KV_HEADS, DIM)
        self.ws = qgemv.AttnWorkspace(1, Q_HEADS, DIM)
        # one sequence, its pages in any order
        self.table = torch.randperm(pages, device="cuda", dtype=torch.int32)[None]

    def project(self, x):
        """q (fp16), k and v (fp32) of x [n, HIDDEN] as [n, heads, DIM]; k and v are slices of the product."""
        y = torch.cat([self.qkv.gemv(part) for part in x.split(16)]).unflatten(1, (-1, DIM))
        return y[:, :Q_HEADS].half(), y[:, Q_HEADS:Q_HEADS + KV_HEADS], y[:, Q_HEADS + KV_HEADS:]

    def slots(self, positions):
        return self.table[0, positions // PAGE].long() * PAGE + positions % PAGE

    def output(self, attended, residual):
        """residual + o product, in calls of at most 16 rows."""
        y = torch.empty_like(residual)
        for lo in range(0, len(residual), 16):
            rows = slice(lo, lo + 16)
            self.o.run_residual(attended[rows].flatten(1).contiguous(), y[rows], residual[rows])
        return y

    def prompt(self, x, past):
        """Tokens x after `past` cached ones: into the cache, and their attention over all of them."""
        n, dev = len(x), x.device
        q, k, v = self.project(x)
        self.cache.write(k, v, self.slots(torch.arange(past, past + n, device=dev)))
        cu_q = torch.tensor([0, n], dtype=torch.int32, device=dev)
        cu_k = torch.tensor([0, past + n], dtype=torch.int32, device=dev)
        keys, values = self.cache.read(self.table, None, cu_k, past + n)  # what later tokens will see
        out, _ = qgemv.attn_prompt(q, keys, values, cu_q, cu_k, max_q=n, workspace=self.ws)
        return self.output(out, x.float())

    def verify(self, x, past, parents):
        """Drafted tokens x, a tree: parents[i] is the draft that i follows, or -1 for the last cached token."""
        n, dev = len(x), x.device
        q, k, v = self.project(x)
        self.cache.write(k, v, self.slots(torch.arange(past, past + n, device=dev)))
        masks = []
        for i, up in enumerate(parents):
            masks.append((masks[up] if up >= 0 else 0) | 1 << i)
        out, _ = self.cache.attend(q, self.table, torch.tensor([past], dtype=torch.int32, device=dev),
                                   torch.tensor([0, n], dtype=torch.int32, device=dev),
                                   torch.tensor(masks, dtype=torch.int64, device=dev), max_ctx=past, max_new=n,
                                   workspace=self.ws)
        return self.output(out, x.float()), (k, v)

    def keep(self, kv, path, past):
        """The accepted drafts become the next positions."""
        at = torch.tensor(path, device="cuda")
        self.cache.write(kv[0][at], kv[1][at], self.slots(torch.arange(past, past + len(path), device="cuda")))


def run(cache="int8"):
    """(largest difference of the accepted drafts' outputs from the same tokens as a prompt, the rms of what the attention
    adds to the residual)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(300, HIDDEN, generator=g, device="cuda").half()
    layer = Layer(cache)
    layer.prompt(x[:200], 0)
    layer.prompt(x[200:290], 200)                     # a second chunk over the first
    # a tree of six drafts: the path 0 - 2 - 4 - 5 is what comes next, 1 and 3 are not
    wrong = torch.randn(2, HIDDEN, generator=g, device="cuda").half()
    drafts = torch.stack([x[290], wrong[0], x[291], wrong[1], x[292], x[293]])
    y, kv = layer.verify(drafts, 290, [-1, -1, 0, 0, 2, 4])
    layer.keep(kv, [0, 2, 4, 5], 290)
    z, _ = layer.verify(x[294:295], 294, [-1])        # plain decoding goes on from there
    layer.ws.status()
    got = torch.cat([y[[0, 2, 4, 5]], z])
    again = Layer(cache)
    want = again.prompt(x[:295], 0)[290:]
    return float((got - want).abs().max()), float((want - x[290:295].float()).square().mean().sqrt())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--cache", choices=sorted(qgemv.KV_FORMATS), default="int8")
    off, rms = run(ap.parse_args().cache)
    print(f"accepted drafts against a prompt: largest difference {off:.2e}, the attention's rms {rms:.3f}")
