"""GPU tests of the prompt attention where rows of a tile share more than their own data: several infinite or NaN values in a
column, and groups of heads that do not fill a tile."""
import itertools
import math

import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]

KINDS = {"float16": torch.float16, "bfloat16": torch.bfloat16}
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def rows(seed, n, heads, d, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, heads, d, generator=g, device="cuda").to(kind)


def attend(q, k, v, nq, nk):
    ws = qgemv.AttnWorkspace(len(nq), q.shape[1], q.shape[2])
    out, lse = qgemv.attn_prompt(q, k, v, cu(nq), cu(nk), max_q=max(nq), workspace=ws)
    torch.cuda.synchronize()
    ws.status()
    return out.double().cpu(), lse.cpu()


def same(got, want):
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(0.5), want.nan_to_num(0.5))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq, nk, one, two", [
    (300, 300, 10, 280),       # in a tile of keys that every row of the later ones sees, and in one that ends inside
    (300, 300, 258, 280),      # in one tile
    (300, 300, 129, 130),
    (40, 5000, 4950, 4990),    # a chunk after a past: few rows, many keys
    (40, 5000, 7, 4990),
])
def test_two_bad_values_in_a_column(kind, d, nq, nk, one, two):
    """A row that sees both has their sum: NaN with any NaN or with infinities of both signs.  (The probabilities of these keys
    are far from 0.)"""
    q, k, v = (rows(i, n, h, d, KINDS[kind]) for i, n, h in ((1, nq, 4), (2, nk, 2), (3, nk, 2)))
    first = torch.arange(nq) + nk - nq          # the last key that each row sees
    for a, b in itertools.product((INF, -INF, NAN), repeat=2):
        v[one, 0, 3], v[two, 0, 3] = a, b
        out, lse = attend(q, k, v, [nq], [nk])
        assert torch.isfinite(lse).all()
        want = torch.zeros(nq, dtype=torch.float64)
        want[first >= one] += a
        want[first >= two] += b
        got = out[:, :2, 3]
        hit = ~torch.isfinite(want)
        assert torch.isfinite(got[~hit]).all()
        for h in range(2):
            assert same(got[hit, h], want[hit]), f"{a} at {one}, {b} at {two}"
        out[:, :2, 3] = 0
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("d", [64, 128])
def test_nan_scores_stay_beside_an_infinite_value(kind, d):
    """A query or a seen key with a NaN gives NaN in every column, the one with an infinite value too."""
    def inputs():
        q, k, v = (rows(i, 300, h, d, KINDS[kind]) for i, h in ((1, 4), (2, 2), (3, 2)))
        v[280, 0, 3] = INF
        return q, k, v
    q, k, v = inputs()
    q[290, 0, 5] = NAN
    out, lse = attend(q, k, v, [300], [300])
    assert torch.isnan(out[290, 0]).all() and torch.isnan(lse[290, 0])
    assert (out[290, 1, 3] == INF) and not torch.isnan(out[290, 1:]).any() and not torch.isnan(out[291:]).any()
    q, k, v = inputs()
    k[10, 0, 5] = NAN
    out, lse = attend(q, k, v, [300], [300])
    assert torch.isnan(out[10:, :2]).all() and torch.isnan(lse[10:, :2]).all()
    assert torch.isfinite(out[:10]).all() and torch.isfinite(out[:, 2:]).all()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("hq, hkv, d, nq, nk", [
    (40, 8, 128, [50] * 20, [1500] * 20),     # groups of 5: 125 rows of a tile of 128
    (5, 1, 128, [50, 9], [3000, 700]),        # shared by several blocks
    (21, 3, 64, [36] * 20, [1500] * 20),      # of 7: 126
    (3, 1, 64, [300], [300]),
])
def test_the_same_bits_whatever_ran_before(kind, hq, hkv, d, nq, nk):
    """Rows of a tile that belong to no query hold what an earlier call left there: here zeros, or values whose scores grow
    along the keys, so that they would move the softmax reference of the rows beside them."""
    dt = KINDS[kind]
    q, k, v = rows(1, sum(nq), hq, d, dt), rows(2, sum(nk), hkv, d, dt), rows(3, sum(nk), hkv, d, dt)
    at = torch.cat([torch.arange(n, device="cuda") for n in nk])
    k[:, :, 0] = (0.02 * at).to(dt)[:, None]
    q[:, :, 0] = 0
    got = []
    for left in (0.0, 64.0, -64.0):
        before = torch.zeros(1024, 64, d, dtype=dt, device="cuda")
        before[:, :, 0] = left
        attend(before, before, before, [1024], [1024])   # 64 heads of their own: every tile of every block is full
        got.append(attend(q, k, v, nq, nk))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


def test_rows_of_other_sequences_do_not_reach_a_result():
    """The rows past the packed queries, and a neighbour's, may hold anything."""
    nq, nk = [30, 20], [700, 900]
    q, k, v = rows(1, 60, 5, 128, torch.float16), rows(2, 1600, 1, 128, torch.float16), rows(3, 1600, 1, 128, torch.float16)
    k[:, :, 0] = (0.02 * torch.arange(1600, device="cuda")).half()[:, None]
    q[:, :, 0] = 0
    want, lse = attend(q, k, v, nq, nk)
    q[50:, :, 0] = 64.0
    out, lse2 = attend(q, k, v, nq, nk)
    assert torch.equal(out[:50], want[:50]) and torch.equal(lse[:50], lse2[:50])
    q[30:50, :, 0] = 64.0
    out, _ = attend(q, k, v, nq, nk)
    assert torch.equal(out[:30], want[:30])


@pytest.mark.parametrize("kind", list(KINDS))
def test_a_bound_of_no_queries_changes_nothing(kind):
    """max_q is a bound that a caller may get wrong: where there are queries, they are answered."""
    q, k, v = (rows(i, 90, 2, 64, KINDS[kind]) for i in (1, 2, 3))
    ws = qgemv.AttnWorkspace(2, 2, 64)
    want, lse = qgemv.attn_prompt(q, k, v, cu([70, 20]), cu([70, 20]), max_q=70, workspace=ws)
    out, lse2 = torch.full_like(want, 5.0), torch.full_like(lse, 5.0)
    qgemv.attn_prompt(q, k, v, cu([70, 20]), cu([70, 20]), max_q=0, workspace=ws, out=out, lse=lse2)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
