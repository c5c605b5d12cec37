"""GPU tests of the key/value cache (qgemv_kv_write, qgemv_kv_read).

The values read back as fp32 must equal the definition's (tests/
attn_reference.py) exactly: codes are decided by fp32 arithmetic that both
sides share by definition, and a code times its scale is one fp32 product.
Read back as fp16 and bf16 they are those values rounded once.
"""
import numpy as np
import pytest

import attn_reference as ref
from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]

FMTS = ["f16", "int8", "q4_0"]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def values(seed, *shape):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape).astype(np.float32) * np.exp(g.standard_normal(shape[-1])).astype(np.float32)
    return x


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def expected(fmt, x):
    return ref.quantised(fmt, x).astype(np.float32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d, heads, page", [(128, 3, 16), (64, 1, 64), (128, 8, 256), (64, 2, 32)])
def test_values_read_back_are_the_definition(fmt, kind, d, heads, page):
    """Tokens in random slots, read back by sequences in the order of their pages; strided k and v."""
    n_pages = 5
    cache = qgemv.KVCache(fmt, n_pages, page, heads, d)
    cache.pages.fill_(0xFF)
    n = n_pages * page - 3
    x = torch.from_numpy(values(d + page, n, 2 * heads + 1, d)).to(TYPES[kind]).cuda()
    k, v = x[:, 1:1 + heads], x[:, 1 + heads:]
    order = np.random.default_rng(1).permutation(n_pages * page)[:n]
    cache.write(k, v, i64(order))
    where = np.full(n_pages * page, -1)
    where[order] = np.arange(n)
    table = np.random.default_rng(2).permutation(n_pages)
    first, second = 2 * page + 5, n_pages * page - 1  # two overlapping views: from 3 on, from 0 on
    cu = [0, first - 3, first - 3 + second]
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        got = cache.read(i32([table, table]), i32([3, 0]), i32(cu), cu[-1], dtype=dt)
        slots = np.array([table[p // page] * page + p % page for p in list(range(3, first)) + list(range(second))])
        src = where[slots]
        keep = src >= 0
        for g, w in zip(got, (k, v)):
            want = torch.from_numpy(expected(fmt, w.float().cpu().numpy()[src[keep]])).to(dt)
            assert torch.equal(g.cpu()[torch.from_numpy(keep)], want)


@pytest.mark.parametrize("fmt", FMTS)
def test_special_vectors(fmt):
    """Zeros, one value, ties, the smallest and largest magnitudes, infinities and NaN."""
    d, f16max = 128, 65504.0
    rows = [np.zeros(d), np.r_[np.zeros(d - 1), 1.0], np.full(d, -2.0), np.tile([1.0, -1.0], d // 2),
            np.tile([-1.0, 1.0], d // 2), np.full(d, 6e-8), np.full(d, f16max), np.arange(d) - 63.5,
            (np.arange(d) % 16 - 8) / 2, np.r_[np.inf, np.zeros(d - 1)], np.r_[np.ones(d - 1), np.nan],
            np.r_[np.ones(d - 1), -np.inf], 127.0 / 2 ** np.arange(d).clip(0, 30)]
    x = np.array(rows, np.float32)[:, None]
    cache = qgemv.KVCache(fmt, 1, 16, 1, d)
    t = torch.from_numpy(x).cuda()
    cache.write(t, -t, i64(range(len(rows))))
    k, v = cache.read(i32([[0]]), None, i32([0, len(rows)]), len(rows), dtype=torch.float32)
    for got, want in ((k, expected(fmt, x)), (v, expected(fmt, -x))):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_other_slots_and_rows_stay(fmt):
    """Slots outside the cache and negative ones are skipped; nothing else of the cache changes; missing pages read zeros;
    rows of no sequence stay; a call of no tokens does nothing."""
    d, heads, page, n_pages = 128, 2, 32, 3
    cache = qgemv.KVCache(fmt, n_pages, page, heads, d)
    x = torch.from_numpy(values(7, n_pages * page, heads, d)).cuda()
    cache.write(x, x, i64(range(n_pages * page)))
    before = cache.pages.clone()
    cache.write(x[:3] + 1, x[:3], i64([-1, n_pages * page, 1 << 40]))
    cache.write(x[:0], x[:0], i64([]))
    assert torch.equal(before, cache.pages)
    cache.write(x[:1] + 1, x[:1], i64([40]))
    table = i32([[1, 5, 0], [-1, 1, 2]])
    out = tuple(torch.full((12, heads, d), 7.0, device="cuda") for _ in range(2))
    k, v = cache.read(table, i32([31, 30]), i32([2, 5, 9]), 12, out=out)
    every = expected(fmt, x.cpu().numpy())
    changed = expected(fmt, (x[:1] + 1).cpu().numpy())[0]
    want = np.full((12, heads, d), 7.0, np.float32)
    want[2], want[3:5] = every[32 + 31], 0          # page 1, then a missing page
    want[5:7], want[7], want[8] = 0, every[32], every[33]
    for got in (k, v):
        assert np.array_equal(got.cpu().numpy(), want)
    k, _ = cache.read(i32([[1]]), i32([8]), i32([0, 1]), 1, dtype=torch.float32)
    assert np.array_equal(k[0].cpu().numpy(), changed)
    k, _ = cache.read(i32([[1]]), i32([-2]), i32([0, 2]), 2)  # positions before the first, and past the table
    assert not k.any()
    k, _ = cache.read(i32([[1]]), i32([32]), i32([0, 2]), 2)
    assert not k.any()


def test_offsets_past_32_bits():
    """A cache of over 4 GB: the last page's first and last slots."""
    d, heads, page = 128, 8, 256
    n_pages = (5 << 30) // (page * heads * d * 4)
    cache = qgemv.KVCache("f16", n_pages, page, heads, d)
    x = torch.from_numpy(values(3, 3, heads, d)).cuda()
    last = (n_pages - 1) * page
    cache.write(x, -x, i64([last, last + page - 1, 0]))
    k, v = cache.read(i32([[n_pages - 1, 0]]), None, i32([0, page + 1]), page + 1, dtype=torch.float32)
    want = expected("f16", x.cpu().numpy())
    assert np.array_equal(k[[0, page - 1, page]].cpu().numpy(), want)
    assert np.array_equal(v[[0, page - 1, page]].cpu().numpy(), -want)


def test_on_another_stream_and_in_a_graph():
    d, heads = 128, 4
    cache = qgemv.KVCache("int8", 4, 16, heads, d)
    x = torch.from_numpy(values(9, 64, heads, d)).cuda()
    y = torch.empty_like(x)
    slots, table, cu = i64(range(64)), i32([[0, 1, 2, 3]]), i32([0, 64])
    out = tuple(torch.empty(64, heads, d, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y.copy_(x)
        cache.write(y, y, slots)
        cache.read(table, None, cu, 64, out=out)
    s.synchronize()
    want = expected("int8", x.cpu().numpy())
    assert np.array_equal(out[0].cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.write(y, y, slots)
        cache.read(table, None, cu, 64, out=out)
    y.copy_(2 * x)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out[1].cpu().numpy(), expected("int8", 2 * x.cpu().numpy()))
