"""GPU tests of the attention of drafted tokens over the cache (qgemv_attn_tree) against its definition in 64 bits on
the values that the cache holds; tolerances are derived in tests/attn_reference.py."""
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
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


class Case:
    """Sequences of ctx cached and new drafted tokens in shuffled pages of a cache whose other bytes are garbage."""

    def __init__(self, fmt, hq, hkv, d, page, ctx, new, seed=0, masks="tree", garbage=0xFF, scale=None, peaky=1.0):
        g = np.random.default_rng(seed + 1000 * d + page)
        self.ctx, self.new, self.hq, self.d, self.fmt, self.page, self.hkv = ctx, new, hq, d, fmt, page, hkv
        self.scale = d ** -0.5 if scale is None else scale
        tot = [c + n for c, n in zip(ctx, new)]
        need = [-(-t // page) for t in tot]
        n_pages = sum(need) + 2
        order = g.permutation(n_pages)
        self.table = np.full((len(ctx), max(need) + 1), -1, np.int64)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.cache = qgemv.KVCache(fmt, n_pages, page, hkv, d)
        self.cache.pages.fill_(garbage)
        self.k = (g.standard_normal((sum(tot), hkv, d)) * peaky).astype(np.float16)
        self.v = g.standard_normal((sum(tot), hkv, d)).astype(np.float16)
        self.q = g.standard_normal((sum(new), hq, d)).astype(np.float16)
        self.start = np.r_[0, np.cumsum(tot)]
        self.cu = np.r_[0, np.cumsum(new)]
        self.masks = []
        for n in new:
            mine = []
            for i in range(n):
                if masks == "chain":
                    mine.append((1 << (i + 1)) - 1)
                elif masks == "none":
                    mine.append(0)
                elif masks == "random":
                    mine.append(int(g.integers(0, 1 << 63)) & ((1 << n) - 1))
                else:
                    up = int(g.integers(max(0, i - 3), i)) if i else -1
                    mine.append((mine[up] if i else 0) | 1 << i)
            self.masks += mine

    def fill(self):
        slots = np.concatenate([[self.table[b][p // self.page] * self.page + p % self.page for p in range(c + n)]
                                for b, (c, n) in enumerate(zip(self.ctx, self.new))])
        self.cache.write(torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda(), i64(slots.astype(np.int64)))
        self.ws = qgemv.AttnWorkspace(len(self.ctx), self.hq, self.d)
        return self

    def run(self, q=None, masks="given", **kw):
        q = torch.from_numpy(self.q).cuda() if q is None else q
        m = None if masks is None else i64([x - (1 << 64) if x >> 63 else x for x in self.masks])
        kw = {"max_ctx": max(self.ctx), "max_new": max(self.new), "workspace": self.ws, "scale": self.scale, **kw}
        out = self.cache.attend(q, i32(self.table), i32(self.ctx), i32(self.cu), m, **kw)
        torch.cuda.synchronize()
        self.ws.status()
        return out

    def reference(self):
        k, v = ref.quantised(self.fmt, self.k), ref.quantised(self.fmt, self.v)
        parts = []
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            see = np.ones((n, c + n), bool)
            for i in range(n):
                see[i, c:] = [(self.masks[self.cu[b] + i] >> j) & 1 for j in range(n)]
            lo, hi = self.start[b], self.start[b + 1]
            parts.append(ref.attention(self.q[self.cu[b]:self.cu[b + 1]].astype(np.float64), k[lo:hi], v[lo:hi], see, self.scale))
        return [np.concatenate(x) for x in zip(*parts)]

    def check(self, name, out, lse):
        ref.check(name, out.float().cpu().numpy(), lse.cpu().numpy(), self.reference())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq, hkv, d, page, ctx, new", [
    (4, 4, 128, 64, [0], [1]),                       # the first token
    (4, 4, 128, 16, [1], [1]),
    (8, 1, 128, 64, [63], [1]),                      # the draft ends a tile
    (8, 1, 64, 16, [64, 15, 16, 0], [1, 1, 1, 1]),
    (5, 1, 128, 32, [300], [16]),                    # 80 rows of a group of 5
    (7, 7, 64, 128, [130, 0, 65], [3, 2, 64]),       # as many drafts as a mask holds
    (16, 2, 128, 256, [700, 3], [9, 16]),
    (6, 2, 128, 16, [1023, 511, 0, 77, 2048], [5, 0, 1, 17, 33]),  # a sequence without drafts
    (64, 8, 128, 64, [2000], [16]),
])
def test_matches_the_definition(fmt, hq, hkv, d, page, ctx, new):
    c = Case(fmt, hq, hkv, d, page, ctx, new).fill()
    c.check(f"{fmt} {ctx} {new}", *c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 2, 3, 5, 6, 7, 8, 9, 11, 13, 16, 17, 25])
def test_tiles_of_rows(fmt, d, new):
    """Numbers of rows (four a token) at and around the ends of the kernels' tiles, in contexts that are split."""
    c = Case(fmt, 4, 1, d, 32, [1500, 0, 333], [new, 1, max(1, new - 2)]).fill()
    c.check(f"{fmt} {d} {new}", *c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("masks", ["chain", "random", "none"])
def test_masks(fmt, masks):
    """Chains (also as no masks at all), any bits, and rows that see nothing but the past (with no past: nothing)."""
    c = Case(fmt, 8, 2, 128, 32, [200, 0, 33], [16, 40, 1], masks=masks).fill()
    out, lse = c.run()
    c.check(masks, out, lse)
    if masks == "chain":
        plain, plain_lse = c.run(masks=None)
        assert torch.equal(plain, out) and torch.equal(plain_lse, lse)
    if masks == "none":
        empty = slice(c.cu[1], c.cu[2])
        assert not out[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_long_contexts_split(fmt):
    """Contexts that the kernel splits, far apart in length, and scores that grow along them."""
    c = Case(fmt, 8, 2, 128, 64, [9000, 70, 4097], [2, 3, 1], peaky=3.0)
    c.k[:, :, :8] += (np.arange(len(c.k)) / 1500.0)[:, None, None].astype(np.float16)
    c.fill()
    c.check("long", *c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_scales(fmt, scale):
    c = Case(fmt, 4, 2, 64, 16, [100], [5], scale=scale).fill()
    c.check(f"scale {scale}", *c.run())


@pytest.mark.parametrize("fmt", ["int8", "q4_0"])
@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_value_magnitudes(fmt, size):
    """Values far from 1: the probabilities meet codes, so fp16's range does not limit them."""
    c = Case(fmt, 4, 1, 128, 32, [300], [4], seed=5)
    c.v = (c.v.astype(np.float32) * size).astype(np.float32)
    g = np.random.default_rng(3)
    c.v *= np.exp(2 * g.standard_normal(c.v.shape[:2] + (1,))).astype(np.float32) if size < 1 else np.float32(1) / 8
    c.k = c.k.astype(np.float32)
    c.fill()
    out, lse = c.run()
    r = c.reference()
    # the smallest results are fp16 subnormals: half a step of 2^-24, which the bound has
    ref.check("sizes", out.float().cpu().numpy(), lse.cpu().numpy(), r)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_what_is_not_seen_stays_out(fmt, bad):
    """A drafted token with infinite or NaN keys or values reaches the rows that see it, and no others; nor does what is in
    the cache past the sequence's end, or in missing pages."""
    for garbage in (0xFF, 0x7C, 0x00):
        c = Case(fmt, 8, 2, 128, 32, [40, 7], [9, 5], garbage=garbage)
        hit = c.start[0] + 40 + 3  # drafted token 3 of sequence 0
        c.v[hit, 0, 5] = bad
        c.v[hit + 1, 1, 77] = bad
        c.fill()
        out, lse = c.run()
        # infinities turn the vector (or group of 32) of a quantised cache to NaN: compare where the reference is finite
        r = c.reference()
        ref.check("unseen", out.float().cpu().numpy(), lse.cpu().numpy(), r)
        sees3 = [(m >> 3) & 1 for m in c.masks[:9]]
        assert any(sees3) and not all(sees3)
        # keys
        c = Case(fmt, 8, 2, 128, 32, [40, 7], [9, 5], garbage=garbage)
        c.k[hit, 0, 5] = bad
        c.fill()
        out, lse = c.run()
        blind = [i for i in range(14) if i >= 9 or not (c.masks[i] >> 3) & 1]
        c.k[hit] = 0
        want = c.reference()
        ref.check("unseen key", out[blind].float().cpu().numpy(), lse[blind].cpu().numpy(), [x[blind] for x in want])


@pytest.mark.parametrize("fmt", FMTS)
def test_missing_pages_are_not_seen(fmt):
    c = Case(fmt, 4, 2, 64, 16, [100], [3]).fill()
    table = c.table.copy()
    c.table[0, 2], c.table[0, 4] = -1, 10 ** 6
    out, lse = c.run()
    k, v = ref.quantised(fmt, c.k), ref.quantised(fmt, c.v)
    see = np.ones((3, 103), bool)
    for i in range(3):
        see[i, 100:] = [(c.masks[i] >> j) & 1 for j in range(3)]
    see[:, 32:48] = see[:, 64:80] = False
    ref.check("missing", out.float().cpu().numpy(), lse.cpu().numpy(), ref.attention(c.q.astype(np.float64), k, v, see, c.scale))
    c.table = table[:, :2]  # a table that ends before the sequence does
    out, lse = c.run()
    see[:, 32:] = False
    ref.check("short table", out.float().cpu().numpy(), lse.cpu().numpy(), ref.attention(c.q.astype(np.float64), k, v, see, c.scale))


def test_strides_hints_streams_and_bits():
    """q and out inside larger rows and head-major; wrong hints change nothing but the split; another stream; the same bits
    each time; nothing outside of out is written."""
    c = Case("int8", 8, 2, 128, 64, [900, 33], [4, 9]).fill()
    want, lse = c.run()
    again, _ = c.run()
    assert torch.equal(want, again)
    wide = torch.full((13, 12, 128), 3.0, dtype=torch.float16, device="cuda")
    wide[:, :8] = torch.from_numpy(c.q).cuda()
    out = torch.full((13, 20, 128), 9.0, dtype=torch.float16, device="cuda")
    got, _ = c.run(q=wide[:, :8], out=out[:, 4:12])
    assert torch.equal(got, want) and (out[:, :4] == 9).all() and (out[:, 12:] == 9).all()
    major = torch.from_numpy(c.q).cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(c.run(q=major)[0], want)
    for hint in ({"max_ctx": 0, "max_new": 0}, {"max_ctx": 10 ** 6, "max_new": 64}, {"max_ctx": 5, "max_new": 1}):
        got, got_lse = c.run(**hint)
        c.check(str(hint), got, got_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = c.run()
    s.synchronize()
    assert torch.equal(got, want)
    for given in (s, s.cuda_stream):
        got, _ = c.run(stream=given)
        s.synchronize()
        assert torch.equal(got, want)


def test_in_a_graph_with_other_lengths():
    """A captured call follows the lengths, tables and masks on the device."""
    c = Case("f16", 4, 2, 128, 32, [500, 64], [3, 2]).fill()
    q, table, ctx, cu = torch.from_numpy(c.q).cuda(), i32(c.table), i32(c.ctx), i32(c.cu)
    masks = i64(c.masks)
    out, lse = torch.empty_like(q), torch.empty(5, 4, device="cuda")
    kw = {"max_ctx": 500, "max_new": 3, "workspace": c.ws, "scale": c.scale, "out": out, "lse": lse}
    c.cache.attend(q, table, ctx, cu, masks, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.attend(q, table, ctx, cu, masks, **kw)
    g.replay()
    torch.cuda.synchronize()
    c.check("graph", out, lse)
    ctx.copy_(i32([100, 64]))  # the first 100 positions, then positions 100 .. 102 as the drafts
    g.replay()
    torch.cuda.synchronize()
    c.ws.status()
    c.k = np.concatenate([c.k[:103], c.k[c.start[1]:]])
    c.v = np.concatenate([c.v[:103], c.v[c.start[1]:]])
    c.ctx, c.start = [100, 64], np.array([0, 103, 169])
    c.check("graph, shorter", out, lse)


def test_more_drafts_than_a_mask_holds_are_left():
    c = Case("f16", 2, 2, 64, 16, [10], [64], masks="chain").fill()
    q = torch.from_numpy(np.concatenate([c.q, c.q[:3]])).cuda()
    out = torch.full_like(q, 5.0)
    masks = i64([x - (1 << 64) if x >> 63 else x for x in c.masks] + [0] * 3)
    got, _ = c.cache.attend(q, i32(c.table), i32([10]), i32([0, 67]), masks, max_ctx=10, max_new=67, workspace=c.ws,
                            out=out, scale=c.scale)
    r = c.reference()
    assert (got[64:] == 5).all()
    assert (np.abs(got[:64].float().cpu().numpy() - r[0]) <= r[2]).all()


def test_offsets_past_32_bits():
    """A sequence whose pages lie past 4 GB of the cache."""
    d, hkv, page = 128, 8, 256
    n_pages = (5 << 30) // (page * hkv * d * 4)
    cache = qgemv.KVCache("f16", n_pages, page, hkv, d)
    g = np.random.default_rng(0)
    k, v = (g.standard_normal((300, hkv, d)).astype(np.float16) for _ in range(2))
    q = g.standard_normal((1, hkv, d)).astype(np.float16)
    table = [n_pages - 1, n_pages - 3]
    slots = [table[p // page] * page + p % page for p in range(300)]
    cache.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), i64(slots))
    out, lse = cache.attend(torch.from_numpy(q).cuda(), i32([table]), i32([299]), i32([0, 1]), None, max_ctx=299, max_new=1,
                            workspace=qgemv.AttnWorkspace(1, hkv, d))
    r = ref.attention(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), np.ones((1, 300), bool), d ** -0.5)
    ref.check("far pages", out.float().cpu().numpy(), lse.cpu().numpy(), r)


def test_status_reports_a_wait_that_ran_out():
    """The kernels record such a wait in the workspace's first word (here the test does); it is reported once."""
    ws = qgemv.AttnWorkspace(2, 8, 128)
    ws.status()
    ws.buffer[:4].copy_(torch.tensor([32, 0, 0, 0], dtype=torch.uint8))
    with pytest.raises(qgemv.QgemvError, match="bounded wait") as e:
        ws.status()
    assert e.value.code == qgemv.QGEMV_ERR_TIMEOUT
    ws.status()
    ws.reset()
    ws.status()
