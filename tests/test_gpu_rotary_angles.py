"""GPU tests of the rotary angle (qgemv_rope_rows): rounded once to fp32, however small it is, and opposite for -position.

Rows (1, 0) turn to (cos, sin).  A small angle's sine is off, relative to itself, by the angle's rounding, 2^-24, sincospif's two
units in the last place, 2^-22, and what |position| 2^-65 turns are of it, below 2^-40 here; times 1 and plus 0 it is not rounded
again."""
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


def turned(freqs, positions):
    """(cos, sin) fp32 [positions, frequencies]."""
    n = len(freqs)
    x = torch.zeros(len(positions), 1, 128, device="cuda")
    x[..., :n] = 1
    r = qgemv.Rotary(128, [n], freqs=freqs)
    y = r.rotate(x, torch.tensor(positions, dtype=torch.int32, device="cuda")[:, None])[:, 0].cpu().double().numpy()
    return y[:, :n], y[:, n:2 * n]


def test_small_angles_keep_their_bits():
    freqs = [1e6 ** (-j / 64) for j in range(64)]
    positions = [1, 2, 3, 7, 100, 1001]
    for scale in (1.0, 1e-3):
        cos, sin = turned([f * scale for f in freqs], positions)
        angle = np.outer(positions, freqs) * scale
        small = angle < 0.5
        assert small.sum() > 150
        want = np.sin(angle)
        assert np.all(np.abs(sin - want)[small] <= (2.0 ** -24 + 2.0 ** -22 + 2.0 ** -40) * want[small])
        assert np.all(np.abs(cos - np.cos(angle))[small] <= 2.0 ** -21)


def test_opposite_positions_are_opposite_angles():
    g = np.random.default_rng(0)
    positions = np.concatenate([[1, 2, 3], g.integers(1, 1 << 20, 200), [2 ** 31 - 1]]).tolist()
    freqs = [500000.0 ** (-j / 64) for j in range(64)]
    cos, sin = turned(freqs, positions)
    back_cos, back_sin = turned(freqs, [-p for p in positions])
    assert np.array_equal(cos, back_cos) and np.array_equal(sin, -back_sin)
