"""GPU tests of calls on a stream that is not torch's current one: their outputs are memory that no other stream still uses, and
that is not handed out again while one does."""
import pytest

from bit_weight_only_gb300 import build, inputs, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls():
    """name -> (function of an input and a stream that returns its outputs as a tuple, an input, another input)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n, heads, d = 1000, 8, 128                       # 2 MB of fp16: blocks of their own in torch's pool
    x, y = (torch.randn(n, heads, d, generator=g, device="cuda").half() for _ in range(2))
    cu, slots = i32([0, n]), torch.arange(1024, device="cuda")
    cache = qgemv.KVCache("f16", 32, 64, heads, d)
    other = qgemv.KVCache("f16", 32, 64, heads, d)
    for c, r in ((cache, x), (other, y)):
        c.write(r, r, slots[:n])
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    each, one = (torch.arange(n + 1, dtype=torch.int32, device="cuda")[:m] for m in (n, n + 1))  # a token a sequence
    tables = table.expand(n, 16).contiguous()
    ws = qgemv.AttnWorkspace(n, heads, d)
    cb = inputs.cbk_centroids(16)
    w = inputs.cbk_packed(inputs.rng("streams/w"), 1 << 16, 256, 4, inputs.cbk_cell_probs(cb))
    gemv = qgemv.QGemv("cbk4", 1 << 16, 256, w, None, cb)
    return {
        "read": (lambda c, s: c.read(table, None, cu, n, stream=s), cache, other),
        "attend": (lambda q, s: cache.attend(q, tables, each, one, max_ctx=n, max_new=1, workspace=ws, stream=s), x, y),
        "attn_prompt": (lambda q, s: qgemv.attn_prompt(q, x, x, cu, cu, max_q=n, workspace=ws, stream=s), x, y),
        "gemv": (lambda a, s: (gemv.gemv(a, s),), x[:16, 0, :].repeat(1, 2).contiguous(), y[:16, 0, :].repeat(1, 2).contiguous()),
    }


def busy():
    """Some tens of milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(40):
        b = a @ a
    return b


@pytest.mark.parametrize("name", ["read", "attend", "attn_prompt", "gemv"])
@pytest.mark.parametrize("as_number", [False, True])
def test_outputs_are_not_memory_still_in_use(name, as_number):
    """Memory that was freed on the current stream before the work on it is done is no output of another stream's call."""
    fn, a, _ = calls()[name]
    want = [t.clone() for t in fn(a, None)]
    busy()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    fn(a, s)  # whatever is set up once
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want]
    busy()
    for t in old:
        t.fill_(7)
    del old, t
    got = fn(a, s.cuda_stream if as_number else s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", ["read", "attend", "attn_prompt", "gemv"])
def test_outputs_stay_while_the_current_stream_uses_them(name):
    """A result that the current stream still has to read when it is freed is not overwritten by the next call."""
    fn, a, b = calls()[name]
    want = [t.clone() for t in fn(a, None)]
    s = torch.cuda.Stream()
    fn(b, s)
    torch.cuda.synchronize()
    got = fn(a, s)
    s.synchronize()
    busy()
    kept = [t.clone() for t in got]
    del got
    again = fn(b, s)
    torch.cuda.synchronize()
    for g, w in zip(kept, want):
        assert torch.equal(g, w)
    del again


@pytest.mark.parametrize("as_number", [False, True])
def test_a_new_workspace_serves_any_stream(as_number):
    """A workspace is set up when it is there, also for a stream that does not wait for the one it was made on."""
    fn, a, _ = calls()["attn_prompt"]
    want = [t.clone() for t in fn(a, None)]
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(3000, 8, 128, generator=g, device="cuda").half()
    cu = i32([0, 3000])
    ws = qgemv.AttnWorkspace(1, 8, 128)
    whole, _ = qgemv.attn_prompt(q, q, q, cu, cu, max_q=3000, workspace=ws)
    nbytes = ws.nbytes
    torch.cuda.synchronize()
    del ws
    torch.full((nbytes,), 127, dtype=torch.uint8, device="cuda")  # what the next one is made of
    s = torch.cuda.Stream()
    busy()
    ws = qgemv.AttnWorkspace(1, 8, 128)
    out, _ = qgemv.attn_prompt(q, q, q, cu, cu, max_q=3000, workspace=ws, stream=s.cuda_stream if as_number else s)
    torch.cuda.synchronize()
    ws.status()
    assert torch.equal(out, whole)
    assert torch.equal(fn(a, None)[0], want[0])
