"""GPU tests of beam search's choice (qgemv_beam_select) where only the order of its sums tells candidates apart: equal rows have
equal log sums wherever they lie in memory, so that ties go to the lower beam and a view's scores are its copy's, bit for bit."""
import numpy as np
import pytest

from bit_weight_only_gb300 import build, qgemv
from test_gpu_beam import TYPES, draw, select

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("beams, vocab, width", [(4, 50021, 16), (9, 9001, 40), (8, 4097, 64), (3, 1023, 9), (8, 515, 20), (5, 7, 30),
                                                 (2, 300007, 7)])
def test_equal_beams_of_any_alignment(kind, beams, vocab, width):
    """Contiguous rows of an odd number of tokens, which all start at other places of a 16-byte unit: score, then beam, then
    token decide."""
    for seed in range(12):
        x = draw(seed, 1, vocab, kind).expand(beams, -1).contiguous()
        s = torch.full((1, beams), -1.0 - seed, device="cuda")
        out, parents, tokens = (t[0].cpu().numpy() for t in select(x, s, width))
        row = x[0].double().cpu().numpy()
        b, t = np.divmod(np.arange(beams * vocab), vocab)
        best = np.lexsort((t, b, -row[t]))[:width]
        n = len(best)
        assert np.array_equal(parents[:n], b[best]) and np.array_equal(tokens[:n], t[best])
        assert all(len(set(out[:n][row[t[best]] == v])) == 1 for v in set(row[t[best]]))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("vocab", [5003, 512, 513, 2048, 16, 3, 70001])
def test_a_view_is_its_copy(kind, vocab):
    n, beams = 2, 3
    for start in range(9):
        wide = torch.full((n * beams, start + vocab + 5), float("nan"), dtype=TYPES[kind], device="cuda")
        wide[:, start:start + vocab] = draw(start, n * beams, vocab, kind)
        x, s = wide[:, start:start + vocab], -torch.arange(6.0, device="cuda").view(n, beams)
        for a, b in zip(select(x, s, 12), select(x.contiguous(), s, 12)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", list(TYPES))
def test_values_of_every_place(kind):
    """One token far above the others, at every place about the chunks' ends, in rows of every alignment."""
    vocab, places = 1537, [0, 1, 7, 8, 255, 503, 504, 505, 510, 511, 512, 513, 519, 520, 1015, 1023, 1024, 1025, 1535, 1536]
    x = torch.zeros(len(places), vocab, dtype=TYPES[kind], device="cuda")
    for i, p in enumerate(places):
        x[i, p] = 20
    _, parents, tokens = select(x, torch.zeros(len(places), 1, device="cuda"), 2)
    assert tokens[:, 0].tolist() == places and tokens[:, 1].tolist() == [1 if p == 0 else 0 for p in places]
