"""GPU tests of the causal attention over packed prompts (qgemv_attn_prompt) against its definition in 64 bits;
tolerances are derived in tests/attn_reference.py."""
import numpy as np
import pytest

import attn_reference as ref
from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]

KINDS = {"float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, kind, hq, hkv, d, nq, nk=None, seed=0, scale=None, peaky=1.0):
        g = np.random.default_rng(seed + d + sum(nq))
        nk = nq if nk is None else nk
        self.kind, self.nq, self.nk, self.d, self.hq = kind, nq, nk, d, hq
        self.scale = d ** -0.5 if scale is None else scale
        self.cu_q, self.cu_k = np.r_[0, np.cumsum(nq)], np.r_[0, np.cumsum(nk)]
        dt = KINDS[kind]
        self.q = torch.from_numpy(g.standard_normal((sum(nq), hq, d)).astype(np.float32)).to(dt)
        self.k = torch.from_numpy((peaky * g.standard_normal((sum(nk), hkv, d))).astype(np.float32)).to(dt)
        self.v = torch.from_numpy(g.standard_normal((sum(nk), hkv, d)).astype(np.float32)).to(dt)
        self.ws = qgemv.AttnWorkspace(len(nq), hq, d)

    def run(self, q=None, k=None, v=None, **kw):
        q, k, v = (a.cuda() if b is None else b for a, b in ((self.q, q), (self.k, k), (self.v, v)))
        kw = {"max_q": max(self.nq), "scale": self.scale, "workspace": self.ws, **kw}
        out = qgemv.attn_prompt(q, k, v, i32(self.cu_q), i32(self.cu_k), **kw)
        torch.cuda.synchronize()
        self.ws.status()
        return out

    def rows(self, most=40):
        """Some rows of every sequence: the first and last ones, around multiples of 64, and others."""
        g = np.random.default_rng(1)
        got = []
        for b, n in enumerate(self.nq):
            near = {x + y for x in range(0, n + 1, 64) for y in (-1, 0)} | set(range(4)) | {n - 2, n - 1}
            near = sorted(i for i in near if 0 <= i < n)
            if len(near) > most:
                near = sorted(set(near[:4] + near[-4:] + list(g.choice(near, most, replace=False))))
            got += [(b, i) for i in near]
        return got

    def check(self, name, out, lse, rows=None):
        q, k, v = (x.double().numpy() for x in (self.q, self.k, self.v))
        rows = self.rows() if rows is None else rows
        at, parts = [], []
        for b, i in rows:
            lo, hi = self.cu_k[b], self.cu_k[b + 1]
            n = max(0, min(hi - lo, i + 1 + (hi - lo) - self.nq[b]))
            r = self.cu_q[b] + i
            parts.append(ref.attention(q[r:r + 1], k[lo:lo + n], v[lo:lo + n], np.ones((1, n), bool), self.scale, self.kind))
            at.append(r)
        want = [np.concatenate(x) for x in zip(*parts)]
        ref.check(name, out[at].double().cpu().numpy(), lse[at].cpu().numpy(), want)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq, hkv, d, nq, nk", [
    (2, 2, 128, [1], None),
    (4, 1, 64, [2, 1, 0, 3], None),
    (3, 3, 128, [127, 128, 129], None),
    (5, 1, 128, [64, 51, 26], None),                 # a group of 5: rows of several tokens in a tile
    (8, 2, 128, [300, 1, 1, 513], None),
    (16, 2, 64, [257, 40], None),
    (7, 1, 64, [19, 700], None),
    (4, 4, 128, [1100], None),
    (8, 8, 128, [5, 130, 1, 200], [900, 131, 256, 777]),   # chunks after a past
    (4, 2, 128, [40, 300, 7], [17, 0, 3]),           # fewer keys than queries: rows that see nothing
    (40, 8, 128, [33, 257], [290, 257]),
    (71, 1, 64, [5, 1], None),                       # one token's heads to a tile
    (128, 1, 128, [3], [130]),
])
def test_matches_the_definition(kind, hq, hkv, d, nq, nk):
    c = Case(kind, hq, hkv, d, nq, nk)
    out, lse = c.run()
    c.check(f"{kind} {nq} {nk}", out, lse)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq, hkv, d, nq, nk", [
    (4, 2, 128, [40, 7], [5000, 3333]),              # few rows, many keys: cut along the keys
    (1, 1, 64, [2500], None),
    (5, 1, 128, [300, 2, 30], [4100, 1, 9000]),      # parts that have no keys
    (2, 1, 128, [1300, 900], [1300, 0]),
])
def test_few_rows_many_keys(kind, hq, hkv, d, nq, nk):
    c = Case(kind, hq, hkv, d, nq, nk)
    out, lse = c.run()
    c.check(f"{kind} {nq} {nk}", out, lse)
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # an infinite value among many keys, seen by the rows from its position on
    c.v[c.nk[0] - 3, 0, 5] = float("inf")
    out, _ = c.run()
    got = torch.isinf(out[:c.nq[0], 0, 5]).cpu()
    assert torch.equal(got, torch.arange(c.nq[0]) >= c.nq[0] - 3)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq, hkv, d, nq, nk", [
    (8, 1, 128, [3, 1, 0, 40] * 11, [4000, 3, 700, 6000] * 11),          # more sequences than lanes; one without queries
    (5, 5, 64, [26, 130, 1, 51], [9000, 130, 20, 51]),
    (64, 8, 128, [16], [9001]),
    (16, 1, 64, [1, 700, 2], [12000, 700, 0]),                           # and one without keys
])
def test_uneven_pieces(kind, hq, hkv, d, nq, nk):
    """Few pieces of very different lengths, which several blocks share."""
    c = Case(kind, hq, hkv, d, nq, nk)
    out, lse = c.run()
    c.check(f"{kind} {nq} {nk}", out, lse)
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_rows_that_see_nothing():
    c = Case("float16", 4, 2, 64, [40, 300], [17, 0])
    out, lse = c.run()
    empty = list(range(23)) + list(range(40, 340))
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()
    assert torch.isfinite(lse[23:40]).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_growing_scores(kind):
    """Scores whose maximum keeps growing along the keys, by more than fp16's range of probabilities, and falling ones."""
    for sign in (1, -1):
        c = Case(kind, 2, 1, 128, [1500], scale=1.0)
        ramp = torch.arange(1500)[:, None] * (sign * 0.25)
        c.k = torch.zeros_like(c.k)
        c.k[:, 0, :4] = (ramp / 4).to(c.k.dtype)
        c.q = torch.zeros_like(c.q)
        c.q[:, :, :4] = 1.0
        out, lse = c.run()
        c.check("ramp", out, lse)


@pytest.mark.parametrize("scale", [2.0, -0.2, 0.0])
def test_scales(scale):
    c = Case("float16", 4, 2, 128, [200, 33], scale=scale)
    c.check(f"scale {scale}", *c.run())


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_seen_stays_out(kind, bad, d):
    """Infinite or NaN keys and values reach the rows that see them, and neither the rows before them nor the sequences next
    to theirs, in whatever tile they meet."""
    nq = [100, 300, 140, 1]
    for b, i in ((1, 130), (1, 299), (2, 0), (0, 99), (3, 0)):
        c = Case(kind, 4, 2, d, nq)
        hit = int(c.cu_k[b]) + i
        c.v[hit, 0, 3] = bad
        c.v[hit, 1, d - 1] = bad
        out, lse = c.run()
        got = out.double().cpu().numpy()
        fine = np.ones(got.shape, bool)
        lo, hi = c.cu_q[b] + i, c.cu_q[b + 1]
        fine[lo:hi, :2, 3] = fine[lo:hi, 2:, d - 1] = False
        assert np.array_equal(np.isfinite(got), fine), f"{b} {i}"
        if not np.isnan(bad):
            assert (got[~fine] == bad).all() or np.isnan(got[~fine][got[~fine] != bad]).all()
        c.v[hit, 0, 3] = c.v[hit, 1, d - 1] = 0
        rows = [(s, r) for s, r in c.rows() if s != b or r < i]
        c.check("values", out, lse, rows)
        c.k[hit, 0, 3] = bad
        out, lse = c.run()
        c.k[hit, 0, 3] = 0
        c.check("keys", out, lse, rows)


def test_strides_streams_and_bits():
    """q, k and v as slices of one stacked product, and head-major; out inside larger rows; another stream; the same bits."""
    c = Case("float16", 6, 2, 128, [150, 9, 260])
    want, lse = c.run()
    assert torch.equal(c.run()[0], want)
    n = sum(c.nq)
    stack = torch.zeros(n, 10, 128, dtype=torch.float16, device="cuda")
    stack[:, :6], stack[:, 6:8], stack[:, 8:] = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out = torch.full((n, 9, 128), 4.0, dtype=torch.float16, device="cuda")
    got, got_lse = c.run(stack[:, :6], stack[:, 6:8], stack[:, 8:], out=out[:, 1:7])
    assert torch.equal(got, want) and torch.equal(got_lse, lse)
    assert (out[:, 0] == 4).all() and (out[:, 7:] == 4).all()
    major = [x.cuda().transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v)]
    assert torch.equal(c.run(*major)[0], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = c.run()
    s.synchronize()
    assert torch.equal(got, want)


def test_rows_past_the_sequences_stay_and_empty_calls():
    c = Case("bfloat16", 2, 2, 64, [70, 20])
    q = torch.cat([c.q, c.q[:9]]).cuda()
    out = torch.full_like(q, 6.0)
    got, _ = c.run(q=q, out=out)
    assert (got[90:] == 6).all()
    c.check("first rows", got, _)
    none, lse = qgemv.attn_prompt(q[:0], c.k[:0].cuda(), c.v[:0].cuda(), i32([0, 0]), i32([0, 0]), max_q=0, workspace=c.ws)
    assert none.shape == (0, 2, 64) and lse.shape == (0, 2)


def test_in_a_graph_with_other_lengths():
    c = Case("float16", 4, 4, 128, [200, 56])
    q, k, v = (x.cuda() for x in (c.q, c.k, c.v))
    cu = i32(c.cu_q)
    out, lse = torch.empty_like(q), torch.empty(256, 4, device="cuda")
    g = torch.cuda.CUDAGraph()
    kw = {"max_q": 256, "workspace": c.ws, "out": out, "lse": lse}
    qgemv.attn_prompt(q, k, v, cu, cu, **kw)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        qgemv.attn_prompt(q, k, v, cu, cu, **kw)
    for nq in ([200, 56], [3, 253], [256, 0]):
        cu.copy_(i32(np.r_[0, np.cumsum(nq)]))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c.nq = c.nk = nq
        c.cu_q = c.cu_k = np.r_[0, np.cumsum(nq)]
        c.check(f"graph {nq}", out, lse)
    c.ws.status()


def test_large_offsets():
    """Token strides that put the last rows past 2^31 elements."""
    n, stride = 70, 1 << 25
    buf = torch.empty(n * stride, dtype=torch.float16, device="cuda")
    c = Case("float16", 2, 1, 64, [n])
    view = buf.view(n, stride)
    parts = [view[:, i * 128:(i + 1) * 128] for i in range(3)]
    q, k, v = parts[0].unflatten(1, (2, 64)), parts[1][:, :64].unflatten(1, (1, 64)), parts[2][:, :64].unflatten(1, (1, 64))
    for dst, src in ((q, c.q), (k, c.k), (v, c.v)):
        dst.copy_(src.cuda())
    out, lse = c.run(q, k, v)
    c.check("far rows", out, lse)
