"""GPU tests of beam search's choice (qgemv_beam_select).

Candidates of one beam are in the order of their logits, exactly, with ties to the lower token.  Scores of different beams are
compared as sums in 64 bits that hold the beams' log sums, which are fp32 sums of exponentials.  Chunks of 512 values: a lane adds
16 of them and lanes are joined five times, fewer than 17 roundings of 2^-24 a chunk; a lane of the beam's warp adds every 32nd
chunk, with a rescaling every eighth one, and five joins follow.  ``off_of`` allows 17 for every 4096 values and 60 more, which is
not less for any vocabulary; exponentials and rescalings are off by 2^-21 each, generously, twice nested: 2^-20.  So a log sum is
off by at most (17 (vocab / 4096 + 2) + 60) 2^-24 + 2^-20; a score's rounding adds 2^-24 of it.
"""
import numpy as np
import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def select(logits, scores, width, **kw):
    n, b = scores.shape
    ws = kw.pop("workspace", None) or qgemv.BeamWorkspace(n, b, logits.shape[1], width)
    return qgemv.beam_select(logits, scores, width, workspace=ws, **kw)


def off_of(vocab):
    return (17 * (vocab / 4096 + 2) + 60) * 2.0 ** -24 + 2.0 ** -20


def check(logits, scores, width, got):
    """Every place against the definition in 64 bits; what a log sum's error could exchange may be exchanged, nothing else."""
    x = logits.detach().cpu().double().numpy()
    s = scores.cpu().double().numpy()
    n, beams = s.shape
    vocab = x.shape[1]
    out, parents, tokens = (t.cpu().numpy() for t in got)
    assert out.shape == parents.shape == tokens.shape == (n, width)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = x.max(1)
        lse = np.where(np.isneginf(top), -np.inf, top + np.log(np.exp(x - np.where(np.isfinite(top), top, 0)[:, None]).sum(1)))
        base = s - lse.reshape(n, beams)
    tol = off_of(vocab)
    for i in range(n):
        lists = []
        for b in range(beams):
            if not np.isfinite(base[i, b]):
                lists.append([])
                continue
            row = x[i * beams + b]
            order = np.lexsort((np.arange(vocab), -row))[:width]
            lists.append([(t, base[i, b] + row[t]) for t in order if row[t] > -np.inf])
        total = sum(map(len, lists))
        at = [0] * beams
        last = None
        for w in range(width):
            if w >= total:
                assert out[i, w] == -np.inf and parents[i, w] == -1 and tokens[i, w] == -1
                continue
            b = parents[i, w]
            assert 0 <= b < beams and at[b] < len(lists[b])
            t, score = lists[b][at[b]]
            assert tokens[i, w] == t, "a beam's candidates come in its own order"
            at[b] += 1
            assert abs(out[i, w] - score) <= tol + 2.0 ** -24 * abs(score)
            best = max(l[a][1] for l, a in zip(lists, [a - (j == b) for j, a in enumerate(at)]) if a < len(l))
            assert score >= best - 2 * tol, "a better candidate was left"
            if last is not None and last[1] == score and lists[last[0]] and x[i * beams + b].tobytes() == x[i * beams + last[0]].tobytes():
                assert (last[0], last[2]) < (b, t), "ties go to the lower beam and token"
            last = b, score, t


def draw(seed, rows, vocab, kind="f32", scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g, device="cuda") * scale).to(TYPES[kind])


def beams_of(seed, n, b):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return -3 * torch.rand(n, b, generator=g, device="cuda")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n, beams, vocab, width", [(1, 1, 1, 1), (1, 1, 5, 8), (1, 4, 32000, 8), (3, 5, 4096, 10), (2, 3, 4097, 64),
                                                    (2, 64, 777, 64), (1, 33, 9001, 40), (7, 2, 50021, 4), (1, 2, 300007, 16),
                                                    (40, 8, 12345, 16), (300, 3, 100, 6), (2, 1, 8191, 33)])
def test_against_the_definition(kind, n, beams, vocab, width):
    x, s = draw(vocab + n, n * beams, vocab, kind), beams_of(n, n, beams)
    check(x, s, width, select(x, s, width))


@pytest.mark.parametrize("kind", list(TYPES))
def test_ties(kind):
    """Equal logits, rows and scores: the lower beam, then the lower token."""
    x = torch.zeros(4, 9000, dtype=TYPES[kind], device="cuda")
    s = torch.zeros(1, 4, device="cuda")
    out, parents, tokens = select(x, s, 64)
    assert bool((parents == 0).all()) and torch.equal(tokens[0].long(), torch.arange(64, device="cuda"))
    x[:, 8000:8003] = 2.0
    out, parents, tokens = select(x, s, 16)
    assert parents[0].tolist() == [0] * 3 + [1] * 3 + [2] * 3 + [3] * 3 + [0] * 4
    assert tokens[0].tolist() == [8000, 8001, 8002] * 4 + [0, 1, 2, 3]
    x = (torch.arange(30000, device="cuda") // 7 % 3).to(TYPES[kind])[None].repeat(2, 1)  # plateaus
    s = torch.tensor([[0.0], [-1.0]], device="cuda")
    out, parents, tokens = select(x, s, 40)
    want = torch.nonzero(x[0] == 2)[:40, 0].int()
    assert torch.equal(tokens[0], want) and torch.equal(tokens[1], want)


@pytest.mark.parametrize("width", [1, 64])
def test_every_order_of_the_logits(width):
    """Rising and falling rows, where every tile holds only better or only worse values; the best at a row's ends."""
    up = torch.arange(100000, device="cuda", dtype=torch.float32) * 1e-3
    x = torch.stack([up, up.flip(0), up.roll(1), up.view(100, 1000).t().reshape(-1)])
    s = torch.tensor([[0.0, -0.5], [-0.25, -0.125]], device="cuda")
    check(x, s, width, select(x, s, width))
    few = torch.full((2, 70000), -5.0, device="cuda")
    few[0, [0, 69999, 4095, 4096]] = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    s = torch.zeros(1, 2, device="cuda")
    check(few, s, width, select(few, s, width))


def test_signed_zeros_are_equal():
    x = torch.full((1, 6000), -1.0, device="cuda")
    x[0, [10, 20, 30, 40]] = torch.tensor([-0.0, 0.0, -0.0, 0.0], device="cuda")
    _, _, tokens = select(x, torch.zeros(1, 1, device="cuda"), 4)
    assert tokens[0].tolist() == [10, 20, 30, 40]


@pytest.mark.parametrize("kind", list(TYPES))
def test_masked_logits_and_dead_beams(kind):
    """-infinity for tokens that are not allowed, also all or all but one; beams that are not in use; rows that hold NaN or
    +infinity give nothing, and nothing of them reaches the others."""
    x = draw(1, 9, 10000, kind)
    x[0] = -float("inf")
    x[1] = -float("inf")
    x[1, 7777] = -30.0
    x[2, 5] = float("nan")
    x[3, 9999] = float("inf")
    x[4, ::2] = -float("inf")
    lowest = torch.finfo(TYPES[kind]).min
    x[5] = lowest
    x[5, 3] = 0
    s = beams_of(2, 1, 9)
    s[0, 6], s[0, 7], s[0, 8] = -float("inf"), float("nan"), float("inf")
    got = select(x, s, 12)
    check(x, s, 12, got)
    assert not set(got[1][0].tolist()) & {0, 2, 3, 6, 7, 8}
    x[5] = lowest
    x[4] = -float("inf")
    got = select(x[:5], s[:, :5], 4)
    assert got[1][0].tolist() == [1, -1, -1, -1] and got[2][0].tolist() == [7777, -1, -1, -1]
    assert torch.isneginf(got[0][0, 1:]).all() and abs(float(got[0][0, 0]) - float(s[0, 1])) < 1e-5
    got = select(x[5:6], s[:, 5:6], 4)        # a row of the lowest value alone: all tokens alike
    assert got[2][0].tolist() == [0, 1, 2, 3]
    s[:] = -float("inf")
    got = select(x, s, 3)
    assert bool((got[1] == -1).all()) and bool((got[2] == -1).all()) and bool(torch.isneginf(got[0]).all())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("start, pad", [(0, 0), (1, 3), (5, 1), (7, 8)])
def test_rows_of_any_alignment(kind, start, pad):
    """Rows inside wider ones: what lies before and behind them does not count."""
    wide = torch.full((6, start + 5003 + pad), float("nan"), dtype=TYPES[kind], device="cuda")
    wide[:, start:start + 5003] = draw(3, 6, 5003, kind)
    x, s = wide[:, start:start + 5003], beams_of(3, 2, 3)
    got = select(x, s, 9)
    check(x, s, 9, got)
    for a, b in zip(got, select(x.contiguous(), s, 9)):
        assert a.dtype == torch.float32 or torch.equal(a, b)  # (sums in another order)
    same = wide[:1, start:start + 5003].expand(6, -1)   # one row for all beams
    check(same, s, 9, select(same, s, 9))


def test_large_logits_and_scores():
    """No overflow on the way, and fp32 sums that would tie are told apart."""
    x = draw(4, 4, 20000) * 1e37
    s = beams_of(4, 2, 2) * 1e5
    got = select(x, s, 5)
    assert bool(torch.isfinite(got[0]).all())
    x = torch.zeros(2, 1000, device="cuda")
    x[0, 5], x[1, 5] = 1.0, 1.0 + 2 ** -20
    s = torch.tensor([[-1000.0, -1000.0]], device="cuda")   # a step of 2^-14 there
    out, parents, tokens = select(x, s, 2)
    assert parents[0].tolist() == [1, 0] and tokens[0].tolist() == [5, 5] and float(out[0, 0]) == float(out[0, 1])


@pytest.mark.parametrize("size", [1e20, 3e38])
def test_scores_at_the_ends_of_fp32(size):
    """Beams that far scores set apart; a sum past fp32 is infinite as a result, and in its order."""
    x = draw(8, 6, 3000)
    s = torch.tensor([[size, -size, size], [-size, 0.0, -1.0]], device="cuda")
    out, parents, tokens = select(x, s, 12)
    # of the first sequence beams 0 and 2 are alike up to their logits, which vanish beside the scores: ties go to beam 0 and
    # the lower token
    assert bool((parents[0] == 0).all()) and torch.equal(tokens[0], torch.arange(12, dtype=torch.int32, device="cuda"))
    assert bool((out[0] == size).all())
    assert set(parents[1].tolist()) <= {1, 2} and bool(torch.isfinite(out[1]).all())
    check(x[4:6], s[1:, 1:], 12, (out[1:], parents[1:] - 1, tokens[1:]))
    y = x * 0 + 3e38
    y[0, 7] = 3.2e38
    out, parents, tokens = select(y[:1], torch.tensor([[size]], device="cuda"), 2)
    assert tokens[0, 0] == 7 and bool((parents == 0).all())


@pytest.mark.parametrize("n, beams, vocab, width", [(16, 4, 32000, 8), (3, 8, 128000, 16), (2, 32, 32000, 64), (5, 3, 1500, 64),
                                                    (2, 64, 4096, 33)])
@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_beams_far_apart(kind, n, beams, vocab, width):
    """One beam far ahead of the others, as scores drift apart, or the only one, as in a first step: all of the result, or all
    of a beam's values, come from it."""
    x = draw(width, n * beams, vocab, kind, 1.0)
    for gap in (2.0, 5.0, 40.0, float("inf")):
        s = beams_of(width, n, beams) - gap
        s[torch.arange(n), (torch.arange(n) * 7 + beams - 1) % beams] = -0.25
        check(x, s, width, select(x, s, width))


@pytest.mark.parametrize("width", [1, 8, 64])
@pytest.mark.parametrize("vocab", [20000, 400000])
def test_scores_that_fp32_cannot_tell_apart(width, vocab):
    """Far scores: many chunks' best candidates are alike in fp32 and in no order, and not in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(width)
    x = 1 + torch.stack([torch.randperm(vocab, generator=g, device="cuda") for _ in range(2)]).float() * 2.0 ** -23
    s = torch.tensor([[-1000.0], [-70000.0]], device="cuda")
    check(x, s, width, select(x, s, width))


def test_rows_past_32_bits():
    """Rows that start beyond 2^32 bytes and elements."""
    n = 1 << 22
    big = torch.zeros(1100, n, dtype=torch.float16, device="cuda")   # 2^32 elements and more
    x = big[:, 1000:4000]
    x[1099] = draw(5, 1, 3000, "f16")[0]
    s = torch.full((1, 1), -1.0, device="cuda")
    got = select(x[1099:], s, 4)
    check(x[1099:], s, 4, got)
    s = torch.full((1100, 1), -1.0, device="cuda")
    got = select(x, s, 4)
    check(x[1090:], s[1090:], 4, tuple(t[1090:] for t in got))


def test_outputs_streams_and_graphs():
    """Given outputs; a stream of its own; two captured graphs that share a workspace, replayed in turn."""
    x, y = draw(6, 12, 33000), draw(7, 12, 33000)
    s = beams_of(6, 3, 4)
    ws = qgemv.BeamWorkspace(3, 4, 33000, 8)
    want, want2 = select(x, s, 8), select(y, s, 8)
    out = tuple(torch.empty_like(t) for t in want)
    assert select(x, s, 8, workspace=ws, out=out) is out
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for t in out:
        t.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = select(x, s, 8, workspace=ws, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for z in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = select(z, s, 8, workspace=ws)
        graphs.append((g, res))
    for _ in range(3):
        for (g, res), w in zip(graphs, (want, want2)):
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(res, w))
    with pytest.raises(qgemv.QgemvError):
        select(torch.cat([x, x]), torch.cat([s, s]), 8, workspace=ws)   # too small for that
    assert all(t.shape == (0, 8) for t in select(x[:0], s[:0], 8, workspace=ws))
