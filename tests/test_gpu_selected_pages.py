"""GPU tests of attention over selected pages (qgemv_kv_summarize, qgemv_kv_select, qgemv_attn_pages).

Summaries and the choice are whole numbers and single IEEE operations, so they equal the definition's bit for bit; the attention
over a choice is held to the bounds of tests/attn_reference.py."""
import numpy as np
import pytest

import attn_reference as ref
from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
FMTS = ["f16", "int8", "q4_0"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def codes(x):
    """INT8 codes and scale of the last axis, the definition."""
    x = np.asarray(x, np.float32)
    a = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.clip(np.rint((x / a[..., None]).astype(np.float32)), -127, 127)
    return np.where(np.isfinite(q) & (a[..., None] > 0), q, 0).astype(np.int64), a


def summaries(values):
    """values fp32 [pages, tokens, heads, d] -> codes [pages, heads, 2, d], scales."""
    both = np.concatenate([values.max(1), values.min(1)], -1)
    q, a = codes(both)
    bad = ~np.isfinite(values).all((1, 3))
    q[bad], a[bad] = 0, np.nan
    return q.reshape(*q.shape[:-1], 2, -1), a


def choice(q, g, table, ctx, n_select, page, sums, scales):
    """The definition's page table and length of one sequence: q fp16 [tokens, q_heads, d]."""
    hkv, n_pages = scales.shape[1], scales.shape[0]
    whole = ctx // page
    rows, tail = [], (2 * page + 62) // page
    at = [e for e in range(min(whole, len(table))) if 0 <= table[e] < n_pages]
    for h in range(hkv):
        x = q[:, h * g:(h + 1) * g].reshape(-1, q.shape[-1]).astype(np.float64)
        w = np.concatenate([np.maximum(x, 0).sum(0), np.minimum(x, 0).sum(0)]).astype(np.float32)
        w = codes(w)[0] if np.isfinite(x).all() else np.zeros(w.shape, np.int64)
        pages = np.array([table[e] for e in at], np.int64)
        dots = (sums[pages, h].reshape(len(pages), w.size) * w).sum(-1)
        score = (dots.astype(np.float32) * scales[pages, h]).astype(np.float32)
        score = np.where(np.isnan(score), np.inf, score)
        best = sorted(np.lexsort((np.arange(len(at)), -score))[:n_select])
        rows.append([table[at[i]] for i in best] + [int(table[e]) if e < len(table) else -1 for e in range(whole, whole + tail)])
    n = len(best)
    return [r + [-1] * (n_select + tail - len(r)) for r in rows], n * page + ctx % page


def cached(fmt, seed, n_pages, page, hkv, d):
    """A cache with every slot written, and its keys and values as the definition has them."""
    g = np.random.default_rng(seed)
    k = g.standard_normal((n_pages * page, hkv, d)).astype(np.float32) * np.exp(0.5 * g.standard_normal((hkv, d))).astype(np.float32)
    v = g.standard_normal((n_pages * page, hkv, d)).astype(np.float32)
    c = qgemv.KVCache(fmt, n_pages, page, hkv, d)
    c.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.arange(n_pages * page, device="cuda"))
    kk, vv = c.read(torch.arange(n_pages, dtype=torch.int32, device="cuda")[None], None, i32([0, n_pages * page]), n_pages * page, dtype=torch.float32)
    return c, kk.cpu().numpy(), vv.cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page, hkv, d", [(16, 1, 64), (64, 8, 128), (256, 3, 128), (32, 5, 64), (128, 2, 64)])
def test_summaries(fmt, page, hkv, d):
    n_pages = 11
    c, k, _ = cached(fmt, page + d, n_pages, page, hkv, d)
    s = qgemv.KeySummary(c)
    s.codes.fill_(99)
    s.scales.fill_(-5)
    which = [7, 0, 3, -1, n_pages, 2147483647, -2147483648, 10, 3]
    s.update(i32(which))
    q, a = summaries(k.reshape(n_pages, page, hkv, d))
    there = sorted({p for p in which if 0 <= p < n_pages})
    assert np.array_equal(s.codes.cpu().numpy()[there], q[there]) and np.array_equal(s.scales.cpu().numpy()[there], a[there])
    other = [p for p in range(n_pages) if p not in there]
    assert bool((s.codes[other] == 99).all()) and bool((s.scales[other] == -5).all())
    s.update(i32([]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page, d", [(16, 128), (64, 64), (128, 128), (256, 64)])
def test_summaries_of_many_pages(fmt, page, d):
    """So many that a warp takes a page's head alone, and not a multiple of a block's; a page twice; one with a NaN."""
    n_pages = 623
    c, k, _ = cached(fmt, page + d, n_pages, page, 1, d)
    bad = torch.full((1, 1, d), float("nan"), device="cuda")
    c.write(bad, bad, torch.tensor([5 * page + page - 1], device="cuda"))
    k = k.reshape(n_pages, page, 1, d)
    k[5, -1] = np.nan
    s = qgemv.KeySummary(c)
    s.update(torch.cat([torch.randperm(n_pages, device="cuda").int(), i32([3, -1, n_pages])]))
    q, a = summaries(k)
    assert np.array_equal(s.codes.cpu().numpy(), q) and np.array_equal(s.scales.cpu().numpy(), a, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_summaries_of_odd_pages(fmt):
    """Zeros, constants, the largest and smallest values, infinities and NaN."""
    page, d = 16, 64
    rows = torch.zeros(8 * page, 2, d, device="cuda")
    rows[page:2 * page] = 2.5
    rows[2 * page:3 * page] = -1e-7
    rows[3 * page] = 60000.0
    rows[4 * page + 5, 1, 7] = float("inf")
    rows[5 * page + 15, 0, 63] = float("nan")
    rows[6 * page:7 * page] = torch.arange(d, device="cuda") - 31.5
    rows[7 * page + 3, 0, 0] = -float("inf")
    c = qgemv.KVCache(fmt, 8, page, 2, d)
    c.write(rows, rows, torch.arange(8 * page, device="cuda"))
    k, _ = c.read(torch.arange(8, dtype=torch.int32, device="cuda")[None], None, i32([0, 8 * page]), 8 * page, dtype=torch.float32)
    s = qgemv.KeySummary(c)
    s.update(torch.arange(8, dtype=torch.int32, device="cuda"))
    q, a = summaries(k.cpu().numpy().reshape(8, page, 2, d))
    assert np.array_equal(s.codes.cpu().numpy(), q) and np.array_equal(s.scales.cpu().numpy(), a, equal_nan=True)
    assert bool(torch.isnan(s.scales).any())


def batch(seed, lens, new, hq, d, page, n_pages, width=None, gaps=0):
    """Queries and a page table in random order for sequences of these lengths."""
    g = np.random.default_rng(seed)
    most = max(need(n + t, page) for n, t in zip(lens, new)) if width is None else width
    table = np.full((len(lens), most), -1, np.int32)
    for b, (n, t) in enumerate(zip(lens, new)):
        m = min(need(n + t, page), most)
        table[b, :m] = g.permutation(n_pages)[:m]
        for e in g.permutation(max(m - 2, 0))[:gaps]:
            table[b, e] = g.choice([-1, n_pages, -9])
    q = torch.from_numpy(g.standard_normal((sum(new), hq, d)).astype(np.float32)).half().cuda()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return q, table, cu


def need(n, page):
    return -(-n // page)


@pytest.mark.parametrize("fmt, page, hq, hkv, d, lens, new, n_select, gaps", [
    ("f16", 16, 8, 2, 128, [700], [1], 5, 0),
    ("int8", 16, 8, 8, 64, [0, 1, 15, 16, 17, 500], [1, 2, 3, 1, 1, 1], 4, 0),
    ("q4_0", 64, 40, 8, 128, [5000, 64, 6300], [3, 64, 1], 7, 0),
    ("int8", 32, 6, 3, 128, [3000, 2990], [9, 0], 0, 0),            # nothing but the tail
    ("f16", 256, 4, 1, 64, [9000, 255, 256], [1, 1, 1], 1000, 0),    # more than there are
    ("q4_0", 16, 16, 2, 64, [40000], [2], 300, 0),                   # a cluster of blocks
    ("int8", 16, 8, 8, 128, [20000, 17000], [1, 5], 1, 3),           # pages that are missing
    ("f16", 16, 64, 8, 128, [4100] * 3, [1, 1, 2], 64, 5),
])
def test_choice_and_attention(fmt, page, hq, hkv, d, lens, new, n_select, gaps):
    n_pages = max(need(n + t, page) for n, t in zip(lens, new)) + 3
    c, k, v = cached(fmt, 1, n_pages, page, hkv, d)
    q, table, cu = batch(2, lens, new, hq, d, page, n_pages, gaps=gaps)
    s = qgemv.KeySummary(c)
    s.update(torch.arange(n_pages, dtype=torch.int32, device="cuda"))
    pages, got_lens = c.select(q, i32(table), i32(lens), i32(cu), summary=s, n_select=n_select)
    ws = qgemv.AttnWorkspace(len(lens), hq, d)
    out, lse = c.attend_pages(q, pages, got_lens, i32(cu), max_ctx=max(lens), max_new=max(new), workspace=ws)
    ws.status()
    sums, scales = s.codes.cpu().numpy().astype(np.int64), s.scales.cpu().numpy()
    qh = q.cpu().numpy()
    for b, (n, t) in enumerate(zip(lens, new)):
        want, length = choice(qh[cu[b]:cu[b + 1]], hq // hkv, list(table[b]), n, n_select, page, sums, scales)
        assert pages[b].tolist() == want and int(got_lens[b]) == length
        rows = range(cu[b], cu[b + 1]) if t < 10 else [cu[b], cu[b] + 1, cu[b + 1] - 1]
        for h in range(hkv):
            own = np.array(want[h])
            pos = np.arange(length + t)
            there = own[pos // page] >= 0
            slots = np.where(there, own[pos // page], 0) * page + pos % page
            kk, vv = k[slots][:, h:h + 1].astype(np.float64), v[slots][:, h:h + 1].astype(np.float64)
            for r in rows:
                see = there & (pos <= length + r - cu[b])
                heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
                w = ref.attention(qh[r:r + 1, heads].astype(np.float64), kk, vv, see[None], d ** -0.5)
                ref.check(f"row {r} head {h}", out[r:r + 1, heads].cpu().numpy(), lse[r:r + 1, heads].cpu().numpy(), w)


def test_all_pages_are_what_attend_gives():
    """With every page chosen the attention is attend()'s, bit for bit: drafted tokens with masks, narrow and wide kernels."""
    for fmt, new in (("int8", 3), ("f16", 16), ("int8", 40), ("q4_0", 16)):
        lens = [1500, 90, 33]
        c, _, _ = cached(fmt, 3, 100, 16, 2, 128)
        q, table, cu = batch(4, lens, [new] * 3, 8, 128, 16, 100)
        masks = torch.from_numpy(np.random.default_rng(5).integers(0, 1 << 62, len(q))).cuda()
        s = qgemv.KeySummary(c)
        s.update(torch.arange(100, dtype=torch.int32, device="cuda"))
        ws = qgemv.AttnWorkspace(3, 8, 128)
        kw = dict(max_ctx=1500, max_new=new, workspace=ws)
        want = c.attend(q, i32(table), i32(lens), i32(cu), masks, **kw)
        pages, l = c.select(q, i32(table), i32(lens), i32(cu), summary=s, n_select=100)
        assert l.tolist() == lens
        # (a wider table lets the sequences be split as before: the split goes by lengths)
        got = c.attend_pages(q, pages, l, i32(cu), masks, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        every = i32(np.repeat(table[:, None], 2, 1))
        got = c.attend_pages(q, every, i32(lens), i32(cu), masks, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_ties_go_to_the_earlier_pages():
    """Equal pages, and queries of zero or with a NaN: the first ones; a page with NaN comes before all."""
    page, n_pages = 16, 600
    c = qgemv.KVCache("f16", n_pages, page, 1, 64)
    rows = torch.ones(n_pages * page, 1, 64, device="cuda").half()
    rows[333 * page + 4, 0, 9] = float("nan")
    c.write(rows, rows, torch.arange(n_pages * page, device="cuda"))
    s = qgemv.KeySummary(c)
    table = torch.randperm(n_pages, device="cuda").int()[None]
    s.update(table[0].contiguous())
    bad = int((table[0] == 333).nonzero())
    for value in (1.0, -1.0, 0.0, float("nan"), float("inf")):
        q = torch.full((1, 2, 64), value, device="cuda").half()
        pages, lens = c.select(q, table, i32([n_pages * page - 7]), i32([0, 1]), summary=s, n_select=9)
        first = sorted(([bad] if bad < n_pages - 1 else []) + [e for e in range(10) if e != bad][:9 - (bad < n_pages - 1)])
        assert pages[0, 0, :9].tolist() == table[0, first].tolist()
        assert int(lens[0]) == 9 * page + page - 7


def test_selected_rows_do_not_see_what_was_left():
    """Infinities in pages without a summary (whose score is that of zeros) reach nobody while better pages are there."""
    page, d = 32, 128
    c = qgemv.KVCache("int8", 40, page, 2, d)
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn(40 * page, 2, d, generator=g, device="cuda")
    k[:10 * page] = float("nan")
    c.write(k, k, torch.arange(40 * page, device="cuda"))
    s = qgemv.KeySummary(c)
    s.update(torch.arange(10, 40, dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 8, d, generator=g, device="cuda").half()
    pages, lens = c.select(q, torch.arange(40, dtype=torch.int32, device="cuda")[None], i32([40 * page - 3]), i32([0, 1]), summary=s, n_select=20)
    assert int(pages[0, :, :20].min()) >= 10
    ws = qgemv.AttnWorkspace(1, 8, d)
    out, lse = c.attend_pages(q, pages, lens, i32([0, 1]), max_ctx=21 * page, max_new=1, workspace=ws)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


def test_strides_tables_and_lengths():
    """Slices of a stacked product as q; a table that is shorter than the context, or has no entries; lengths below 0; a cu_q
    whose sequences have no rows."""
    c, k, _ = cached("q4_0", 6, 50, 16, 2, 64)
    s = qgemv.KeySummary(c)
    s.update(torch.arange(50, dtype=torch.int32, device="cuda"))
    sums, scales = s.codes.cpu().numpy().astype(np.int64), s.scales.cpu().numpy()
    stack = torch.randn(5, 12, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    q = stack[:, 3:11]
    table, lens, cu = np.arange(30, dtype=np.int32).reshape(3, 10)[:, ::-1].copy(), [160 * 3, 100, -4], [0, 2, 2, 5]
    pages, l = c.select(q, i32(table), i32(lens), i32(cu), summary=s, n_select=4)
    for b in range(3):
        want, length = choice(q.cpu().numpy()[cu[b]:cu[b + 1]], 4, list(table[b]), max(lens[b], 0), 4, 16, sums, scales)
        assert pages[b].tolist() == want and int(l[b]) == length
    again = c.select(q.contiguous(), i32(table), i32(lens), i32(cu), summary=s, n_select=4)
    assert torch.equal(again[0], pages) and torch.equal(again[1], l)
    none = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    pages, l = c.select(q, none, i32(lens), i32(cu), summary=s, n_select=4)
    assert bool((pages == -1).all()) and l.tolist() == [0, 100 % 16, 0]
    pages, l = c.select(q[:0], i32(table), i32(lens), i32([0] * 4), summary=s, n_select=4)
    assert l.tolist() == [64, 64 + 4, 0]


def test_the_longest_tables():
    """A table of as many pages as a call takes, on a cluster of eight blocks, each page in it many times."""
    c, k, _ = cached("q4_0", 7, 3000, 16, 1, 64)
    s = qgemv.KeySummary(c)
    s.update(torch.arange(3000, dtype=torch.int32, device="cuda"))
    table = np.arange(49152, dtype=np.int64) * 7 % 3000
    q = torch.randn(1, 1, 64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    ctx = 49152 * 16
    pages, l = c.select(q, i32(table)[None], i32([ctx]), i32([0, 1]), summary=s, n_select=5000)
    want, length = choice(q.cpu().numpy(), 1, list(table), ctx, 5000, 16, s.codes.cpu().numpy().astype(np.int64), s.scales.cpu().numpy())
    assert pages[0].tolist() == want and int(l[0]) == length == 5000 * 16


def test_streams_and_graphs():
    c, _, _ = cached("int8", 8, 200, 16, 2, 128)
    s = qgemv.KeySummary(c)
    lens = i32([3000])
    q, table, cu = batch(9, [3000], [1], 8, 128, 16, 200)
    q2 = batch(10, [3000], [1], 8, 128, 16, 200)[0]
    fresh, table, cu = torch.arange(200, dtype=torch.int32, device="cuda"), i32(table), i32(cu)
    ws = qgemv.AttnWorkspace(1, 8, 128)

    def step(q, **kw):
        s.update(fresh, **kw)
        pages, l = c.select(q, table, lens, cu, summary=s, n_select=12, **kw)
        return pages, l, *c.attend_pages(q, pages, l, cu, max_ctx=13 * 16, max_new=1, workspace=ws, **kw)
    want, want2 = step(q), step(q2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(q, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = q.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(x)
    for y, w in ((q2, want2), (q, want)):
        x.copy_(y)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
