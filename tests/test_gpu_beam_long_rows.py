"""GPU tests of beam search's log sums (qgemv_beam_select) over rows of up to 2^26 tokens: their error does not grow with the row.

Roundings of 2^-24 on the way of a term: its chunk's sum 6 in a lane and 5 between the lanes, the beam's 4 + 1 + 5, the logarithm
1: 22.  Two exponentials, each within 2^-22: 8.  Their arguments (x - m) log2(e) are rounded twice,
with a rounded constant: 3 |x - m| 2^-24 in the exponent, on the average of the terms by their weight.  Together
(30 + 3 E|x - max|) 2^-24, to first order: a relative error of the sum is the absolute one of its logarithm.  The score adds half a
step."""
import math

import pytest

from bit_weight_only_gb300 import build, qgemv
from test_gpu_beam import TYPES, select

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def check(x):
    """The first place of every row (a beam each of a sequence of its own) against sums in 64 bits."""
    best, _, tokens = select(x, torch.zeros(len(x), 1, device="cuda"), 1)
    for row, score, token in zip(x, best[:, 0].tolist(), tokens[:, 0].tolist()):
        top = float(row.max())
        assert token == int((row == top).nonzero()[0])
        total = far = 0.0
        for part in row.split(1 << 24):
            d = top - part.double()
            e = torch.exp(-d)
            total += float(e.sum())
            far += float((e * torch.where(e > 0, d, 0)).sum())
        want = -math.log(total)
        assert abs(score - want) <= (30 + 3 * far / total) * 1.001 * 2.0 ** -24 + 2.0 ** -24 * abs(want)
        del d, e, part


@pytest.mark.parametrize("kind, vocab", [("f16", 1 << 26), ("bf16", (1 << 25) + 4099), ("f32", 1 << 25), ("f32", 300001)])
def test_chunks_whose_sums_round_one_way(kind, vocab):
    """Each chunk of 512 adds the same, no multiple of what a long sum's last place is."""
    for value in (0.2, 0.7):
        x = torch.zeros(1, vocab, dtype=TYPES[kind], device="cuda")
        x[0, 100::512] = math.log(value)
        check(x)


@pytest.mark.parametrize("kind, vocab", [("f32", 1 << 25), ("f16", 1 << 26), ("f32", 1 << 18)])
def test_rising_rows(kind, vocab):
    """A new largest value in every chunk, and the other way."""
    up = torch.linspace(0, 16, vocab, device="cuda", dtype=torch.float32).to(TYPES[kind])
    check(torch.stack([up, up.flip(0)]))


def test_random_rows():
    g = torch.Generator(device="cuda").manual_seed(1)
    for scale in (0.5, 3.0):
        check((torch.randn(2, 1 << 24, generator=g, device="cuda") * scale))
