"""The README's calls around the paged cache, as they stand there: they run, and every page that is in use afterwards is held by a
row."""
import os
import re

import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def block(call):
    """The Python block that makes this call."""
    found = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if call in b]
    assert len(found) == 1
    return found[0]


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens", [(64, 64, 128), (63, 1, 64), (10, 70, 129)])
def test_a_step_of_beam_search_loses_no_page(lens):
    """Lengths at a page's end, where the new token takes a new page, and others; a parent with two children."""
    page, rows, kv_heads, vocab = 64, 3, 2, 1000
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda").half()  # noqa: E731
    code = block("pool.fork(").replace("pool = qgemv.PagePool(n_pages, 64)", "pool = made")
    made = qgemv.PagePool(40, page)
    table = torch.full((rows, 4), -1, dtype=torch.int32, device="cuda")
    made.reserve(table, i32(0, 0, 0), i32(*lens))
    cache = qgemv.KVCache("int8", 40, page, kv_heads, 128)
    names = dict(qgemv=qgemv, made=made, cache=cache, table=table, lens=i32(*lens), parents=i32(1, 1, 2), n_pages=40, n=1, b=rows,
                 vocab=vocab, width=rows, logits=draw(rows, vocab), scores=torch.zeros(1, rows, device="cuda"), q=draw(rows, 8, 128),
                 k=draw(rows, kv_heads, 128), v=draw(rows, kv_heads, 128), positions=torch.zeros(rows, 3, dtype=torch.int32, device="cuda"),
                 slots=torch.arange(rows, device="cuda") + 39 * page, full_pages=i32(0, 1), ctx_lens=i32(*lens),
                 cu_q=torch.arange(rows + 1, dtype=torch.int32, device="cuda"), ws=qgemv.AttnWorkspace(rows, 8, 128))
    exec(code, names)
    now = [lens[p] + 1 for p in (1, 1, 2)]
    held = [names["table"][r, :-(-n // page)].tolist() for r, n in enumerate(now)]
    assert all(p >= 0 for row in held for p in row)
    counts = torch.bincount(torch.tensor(sum(held, [])), minlength=40).tolist()
    assert made.refs.tolist() == counts
    made.release(names["table"], i32(*now))
    assert not made.refs.any()
