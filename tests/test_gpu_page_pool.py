"""GPU tests of the page pool (qgemv_pool_*) and of page copies (qgemv_kv_copy_pages): whole numbers and bytes, which equal a
plain simulation's."""
import numpy as np
import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def need(n, page):
    return -(-max(int(n), 0) // page)


class Plain:
    """The definition: lists and loops."""

    def __init__(self, n, page):
        self.refs, self.page, self.missing = [0] * n, page, 0

    def give(self):
        for p, r in enumerate(self.refs):
            if r <= 0:
                self.refs[p] = 1
                return p
        self.missing += 1
        return -1

    def ok(self, p):
        return 0 <= p < len(self.refs)

    def reserve(self, table, have, want):
        for b, row in enumerate(table):
            for e in range(need(have[b], self.page), min(need(want[b], self.page), len(row))):
                row[e] = self.give()

    def fork(self, table, parents, lens):
        width = len(table[0]) if len(table) else 0
        new, src, dst, tokens = [], [], [], []
        kids = [[r for r, p in enumerate(parents) if p == b] for b in range(len(table))]
        for b, row in enumerate(table):
            for e in range(min(need(lens[b], self.page), width)):
                part = lens[b] % self.page and e == need(lens[b], self.page) - 1
                if self.ok(row[e]):
                    self.refs[row[e]] += (min(len(kids[b]), 1) if part else len(kids[b])) - 1
        for r, b in enumerate(parents):
            row, s, t = [-1] * width, -1, 0
            if 0 <= b < len(table):
                used = need(lens[b], self.page)
                row[:min(used, width)] = table[b][:min(used, width)]
                if lens[b] > 0 and lens[b] % self.page and used <= width and self.ok(row[used - 1]) and kids[b][0] != r:
                    s, t = row[used - 1], lens[b] % self.page
                    row[used - 1] = None
            new.append(row)
            src.append(s)
            tokens.append(t)
            dst.append(-1)
        for r, row in enumerate(new):
            if None in row:
                dst[r] = row[row.index(None)] = self.give()
        return new, src, dst, tokens

    def release(self, table, lens, keep):
        for b, row in enumerate(table):
            for e in range(need(keep[b], self.page) if keep is not None else 0, min(need(lens[b], self.page), len(row))):
                if self.ok(row[e]):
                    self.refs[row[e]] -= 1
                row[e] = -1

    def compact(self, table):
        used = sum(r > 0 for r in self.refs)
        src = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(used) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        return [[to.get(p, p) for p in row] for row in table], src, dst


def same(pool, plain):
    assert pool.refs.tolist() == plain.refs and int(pool._state[0]) == plain.missing


@pytest.mark.parametrize("n_pages, page, rows, width, seed", [(40, 16, 3, 9, 0), (300, 64, 17, 12, 1), (5000, 16, 64, 40, 2),
                                                              (40000, 128, 300, 100, 3), (17, 256, 5, 8, 4), (16400, 32, 1, 1000, 5)])
def test_a_history_of_calls(n_pages, page, rows, width, seed):
    """Random calls of every kind, one after the other, with lengths of 0, at pages' ends and past the table; pages run out in
    some."""
    g = np.random.default_rng(seed)
    pool, plain = qgemv.PagePool(n_pages, page), Plain(n_pages, page)
    table = [[-1] * width for _ in range(rows)]
    lens = [0] * rows
    dev = i32(table)
    for step in range(12):
        more = [int(n + g.choice([0, 1, page - n % page, g.integers(0, 2 * page), g.integers(0, width * page // 3 + 1)])) for n in lens]
        plain.reserve(table, lens, more)
        pool.reserve(dev, i32(lens), i32(more))
        assert dev.tolist() == table
        same(pool, plain)
        lens = [min(n, width * page) for n in more]
        kind = step % 4
        if kind == 0:
            keep = [int(g.integers(0, n + 1)) for n in lens]
            plain.release(table, lens, keep)
            pool.release(dev, i32(lens), i32(keep))
            lens = keep
        elif kind in (1, 2):
            n_new = rows if kind == 1 else int(g.integers(1, 2 * rows + 1))
            parents = [int(p) for p in g.integers(-1, rows + 1, n_new)]
            table, src, dst, tokens = plain.fork(table, parents, lens)
            dev, s, d, t = pool.fork(dev, i32(parents), i32(lens))
            assert (s.tolist(), d.tolist(), t.tolist()) == (src, dst, tokens)
            lens = [lens[p] if 0 <= p < rows else 0 for p in parents]
            rows = n_new
        else:
            table, src, dst = plain.compact(table)
            dev, s, d = pool.compact(dev)
            k = len(src)
            assert s[:k].tolist() == src and d[:k].tolist() == dst and bool((s[k:] == -1).all()) and bool((d[k:] == -1).all())
        assert dev.tolist() == table
        same(pool, plain)
    if plain.missing:
        with pytest.raises(qgemv.QgemvError, match=f"{plain.missing} pages"):
            pool.status()
    pool.status()
    pool.release(dev, i32([width * page] * rows))
    assert int(pool.refs.clamp(min=0).sum()) == 0 and bool((dev == -1).all())


def test_reserve_edges():
    """Negative and falling lengths give nothing; no rows and no entries are calls like others; a full pool gives -1."""
    pool = qgemv.PagePool(10, 16)
    t = torch.full((3, 4), 77, dtype=torch.int32, device="cuda")
    pool.reserve(t, i32([-5, 30, 0]), i32([1, 10, -3]))
    assert t.tolist() == [[0, 77, 77, 77], [77] * 4, [77] * 4]
    pool.reserve(t[:0], i32([]), i32([]))
    pool.reserve(t[:, :0].contiguous(), i32([0] * 3), i32([9] * 3))
    pool.reserve(t, i32([16, 0, 0]), i32([64, 64, 1 << 30]))
    assert t.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, -1, -1]]
    with pytest.raises(qgemv.QgemvError, match="2 pages"):
        pool.status()
    pool.status()
    one = qgemv.PagePool(1, 16)
    t = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    one.reserve(t, i32([0]), i32([5]))
    new, src, dst = one.compact(t)
    assert new.tolist() == [[0]] and src.numel() == 0


def test_most_rows():
    rows = 4096
    pool = qgemv.PagePool(2 * rows + 5, 16)
    t = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pool.reserve(t, zero, zero + 20)
    assert torch.equal(t.flatten(), torch.arange(2 * rows, dtype=torch.int32, device="cuda"))
    # every row's first child is row 4095 - r, and nobody has a second one
    new, src, dst, tokens = pool.fork(t, torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda"), zero + 20)
    assert torch.equal(new, t.flip(0)) and bool((src == -1).all()) and bool((dst == -1).all())
    # row 0 has all of the children: its whole page is shared, the others' pages are free for the copies
    new, src, dst, tokens = pool.fork(t, zero, zero + 20)
    assert bool((new[:, 0] == 0).all()) and int(pool.refs[0]) == rows and int(new[0, 1]) == 1
    assert torch.equal(new[1:, 1], torch.arange(2, rows + 1, dtype=torch.int32, device="cuda")) and torch.equal(dst[1:], new[1:, 1])
    assert bool((src[1:] == 1).all()) and bool((tokens[1:] == 4).all()) and int(src[0]) == -1
    with pytest.raises(qgemv.QgemvError):
        pool.reserve(torch.full((rows + 1, 1), -1, dtype=torch.int32, device="cuda"), i32([0] * (rows + 1)), i32([1] * (rows + 1)))


@pytest.mark.parametrize("rows, width", [(1, 1), (3, 700), (64, 512), (64, 513), (2, 70001)])
@pytest.mark.parametrize("n_pages", [1, 2, 4095, 4097, 16384, 16385])
def test_packing_of_pools_and_tables_of_any_size(n_pages, rows, width):
    """Counts of no, some and all pages, tables that name pages in any order and more than once, in place and not."""
    g = np.random.default_rng(n_pages + width)
    for used in (0.0, 0.02, 0.6, 1.0):
        pool, plain = qgemv.PagePool(n_pages, 16), Plain(n_pages, 16)
        refs = (g.random(n_pages) < used) * g.integers(1, 5, n_pages)
        plain.refs = refs.tolist()
        pool.refs.copy_(i32(plain.refs))
        table = g.integers(-1, n_pages, (rows, width)).tolist()
        dev = i32(table)
        want, src, dst = plain.compact(table)
        new, s, d = pool.compact(dev, out=dev if used == 0.6 else None)
        assert new.tolist() == want and s[:len(src)].tolist() == src and d[:len(dst)].tolist() == dst
        assert bool((s[len(src):] == -1).all()) and bool((d[len(dst):] == -1).all())
        same(pool, plain)


def test_tables_with_numbers_that_are_no_pages():
    """Entries outside the pool are passed over, and nothing outside the counts is touched."""
    bad = [[-7, 3, 1 << 30], [2, -2147483648, 99], [2147483647, 3, 5]]
    pool = qgemv.PagePool(20, 16)
    pool.refs.fill_(1)
    new, src, dst, tokens = pool.fork(i32(bad), i32([0, 0, 1, 7, -3, 2147483647, -2147483648]), i32([48, 40, 48]))
    assert new.tolist() == [bad[0], bad[0], bad[1], [-1] * 3, [-1] * 3, [-1] * 3, [-1] * 3]
    assert src.tolist() == [-1] * 7 and dst.tolist() == [-1] * 7
    want = [1] * 20
    want[3] = 1  # one more of row 0, one less of row 2
    want[5] = 0
    assert pool.refs.tolist() == want
    t = i32(bad)
    pool.release(t, i32([48] * 3))
    want[3] -= 2
    want[2], want[5] = 0, -1
    assert pool.refs.tolist() == want
    new, src, dst = pool.compact(i32(bad))
    assert new[0, 0] == -7 and new[0, 2] == 1 << 30 and new[2, 0] == 2147483647
    pool.compact(t, out=t)


FMTS = {"f16": 4, "int8": 2, "q4_0": 1}


@pytest.mark.parametrize("fmt", ["f16", "int8", "q4_0"])
@pytest.mark.parametrize("page, heads, d", [(16, 1, 64), (64, 8, 128), (256, 3, 128), (32, 40, 64)])
def test_copies(fmt, page, heads, d):
    """Whole pages, and the first tokens of every head in blocks of 16; other bytes stay; numbers that are no pages are passed
    over."""
    n_pages = 30
    c = qgemv.KVCache(fmt, n_pages, page, heads, d)
    block = c.pages.numel() // n_pages // heads // (page // 16)
    start = torch.randint(0, 256, (n_pages, heads, page // 16, block), dtype=torch.uint8, device="cuda")
    src, dst = [1, 2, -1, 30, 5, 6, 7, 8, 0, 9], [20, 21, 22, 23, -1, 30, 24, 25, 29, 26]
    tokens = [0, 1, 16, 16, 16, 16, 17, page - 1, page, 1 << 30]
    for given in (None, tokens, [-5] * 10):
        c.pages.copy_(start.flatten())
        c.copy_pages(i32(src), i32(dst), None if given is None else i32(given))
        want = start.clone()
        for k, (s, t) in enumerate(zip(src, dst)):
            if 0 <= s < n_pages and 0 <= t < n_pages:
                n = page // 16 if given is None else min(page // 16, need(given[k], 16))
                want[t, :, :n] = start[s, :, :n]
        assert torch.equal(c.pages.view_as(want), want)
    c.copy_pages(i32([]), i32([]))


def test_copied_tokens_read_the_same():
    c = qgemv.KVCache("int8", 8, 64, 2, 128)
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(100, 2, 128, generator=g, device="cuda") for _ in range(2))
    c.write(k, v, torch.arange(100, device="cuda"))
    c.copy_pages(i32([0, 1]), i32([5, 3]), i32([64, 36]))
    cu = i32([0, 100])
    for a, b in zip(c.read(i32([[0, 1]]), None, cu, 100), c.read(i32([[5, 3]]), None, cu, 100)):
        assert torch.equal(a, b)


def test_pages_past_32_bits():
    """Pages beyond 4 GB of a cache."""
    c = qgemv.KVCache("f16", 1200, 256, 32, 128)   # 4 MB each
    assert c.pages.numel() > 1 << 32
    row = c.pages.view(1200, -1)
    row[1199].random_(0, 256)
    row[3].zero_()
    c.copy_pages(i32([1199, 3]), i32([2, 1150]))
    assert torch.equal(row[2], row[1199]) and int(row[1150].sum()) == 0
    row[1100].zero_()
    c.copy_pages(i32([2]), i32([1100]))
    assert torch.equal(row[1100], row[1199])


def test_streams_and_graphs():
    """A step of beam search captured once and replayed on other tables; the pool's counts go on from replay to replay."""
    page, width = 16, 6
    pool, plain = qgemv.PagePool(60, page), Plain(60, page)
    c = qgemv.KVCache("q4_0", 60, page, 1, 64)
    lens = [37, 37, 50, 50]
    table = [[-1] * width for _ in lens]
    t = i32(table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pool.reserve(t, i32([0] * 4), i32(lens), stream=s)
    s.synchronize()
    plain.reserve(table, [0] * 4, lens)
    assert t.tolist() == table
    parents, ln = i32([0, 0, 0, 0]), i32(lens)
    before = pool.refs.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, src, dst, tokens = pool.fork(t, parents, ln)
        c.copy_pages(src, dst, tokens)
        t.copy_(new)
    assert torch.equal(pool.refs, before)
    for p in ([1, 1, 2, 3], [0, 2, 2, 1], [3, 3, 3, 3], [0, 1, 2, 3]):
        parents.copy_(i32(p))
        g.replay()
        table, a, b, n = plain.fork(table, p, lens)
        lens = [lens[x] for x in p]
        assert (t.tolist(), src.tolist(), dst.tolist(), tokens.tolist()) == (table, a, b, n)
        same(pool, plain)
        ln.copy_(i32(lens))
