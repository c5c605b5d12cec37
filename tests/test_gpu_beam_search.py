"""The operators around the cache together, as the beam search of examples/beam_search.py uses them: after forks, copies, pages
given out again and a packing, each beam's cache holds what its own tokens leave there when nothing is shared, and its score is
that of its tokens.

The cache is compared bit for bit: rows of the q|k|v product are the same bits whatever rows are beside them in the
batch-invariant mode, and everything after it works row by row.  The score is compared with a replay of the same tokens alone,
whose attention takes the same cached values; differences are those of fp32 sums in another order (2^-20 of values up to 100 is
the wide bound that is taken for each of the 40 steps' log probabilities, plus the fp16 rounding of the head's inputs, 2^-11 of
sums of 1024 products of about 0.03 * 0.02 in random directions: below 2e-3 each)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from bit_weight_only_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("beam_search", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    real = m.Model.__init__

    def init(self):
        real(self)
        for h in (self.qkv, self.o, self.head):
            h.set_batch_invariant(True)
    m.Model.__init__ = init
    return m


@pytest.mark.parametrize("cache", ["f16", "int8", "q4_0"])
@pytest.mark.parametrize("select", [0, 3])
@pytest.mark.parametrize("beams, steps, prompt", [(5, 40, 100), (16, 20, 17), (1, 3, 2)])
def test_beams_are_their_tokens(example, cache, select, beams, steps, prompt):
    from bit_weight_only_gb300 import qgemv
    search, tokens = example.run(cache, beams, steps, prompt, select)
    n = prompt - 1 + steps
    assert search.length == n and search.history.shape == (beams, steps)
    # the pages in use are the lowest, and no page that a beam writes on is another's
    used = int((search.pool.refs > 0).sum())
    assert bool((search.pool.refs[used:] == 0).all()) and int(search.table.max()) == used - 1
    held = search.table[:, :-(-n // example.PAGE)]
    assert bool((held >= 0).all()) and int(search.pool.refs.sum()) == held.numel()
    if n % example.PAGE:
        last = held[:, -1]
        assert len(set(last.tolist())) == beams and bool((search.pool.refs[last.long()] == 1).all())
    # what the beams share is stored once
    assert used < held.numel() or beams == 1
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    model = search.model
    for b in {0, beams - 1, beams // 2}:
        mine = torch.cat([tokens, search.history[b, :-1]])
        _, q, k, v = model.project(mine)
        alone = qgemv.KVCache(cache, -(-n // example.PAGE), example.PAGE, example.KV_HEADS, example.DIM)
        at = torch.arange(n, device="cuda")
        alone.write_rotated(model.rotary, q, k, v, at[:, None].int(), at)
        pages = torch.arange(alone.n_pages, dtype=torch.int32, device="cuda")[None]
        for x, y in zip(search.cache.read(search.table[b:b + 1].contiguous(), starts, cu, n), alone.read(pages, starts, cu, n)):
            assert torch.equal(x, y)
    # the best beam's score, from its tokens alone
    one = example.Search(model, tokens, 1, steps, cache, select)
    seen = []
    real = qgemv.beam_select

    def watch(logits, *args, **kw):
        seen.append(logits[0].double())
        return real(logits, *args, **kw)
    example.qgemv.beam_select = watch
    try:
        for token in search.history[0]:
            one.step()
            one.tokens = token[None]
    finally:
        example.qgemv.beam_select = real
    total = sum(float(torch.log_softmax(x, 0)[t.long()]) for x, t in zip(seen, search.history[0]))
    assert abs(total - float(search.scores[0, 0])) <= steps * 2e-3
    assert bool((search.scores[0, :-1] >= search.scores[0, 1:]).all())


def test_positions_count(example):
    """The same token at another place gives other keys: the rotation is in the cache."""
    search, tokens = example.run("f16", 2, 3, 40)
    k = search.cache.read(search.table[:1].contiguous(), None, torch.tensor([0, 42], dtype=torch.int32, device="cuda"), 42, dtype=torch.float32)[0]
    _, q, plain, v = search.model.project(tokens[:1])
    assert float((k[0] - plain[0]).abs().max()) <= 2 ** -10 * float(plain.abs().max())     # position 0 turns nothing
    _, q, plain, v = search.model.project(tokens[20:21])
    assert float((k[20] - plain[0]).abs().max()) > 0.1 * float(plain.abs().max())
