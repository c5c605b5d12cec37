"""GPU tests of the cache and of the drafted tokens' attention at the ends of their number ranges; tolerances are derived in
tests/attn_reference.py."""
import numpy as np
import pytest

import attn_reference as ref
from bit_weight_only_gb300 import build, qgemv
from test_gpu_attn_tree import Case, i32, i64

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]

FMTS = ["f16", "int8", "q4_0"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-8, -13, -18])
def test_small_queries(fmt, d, power):
    """Queries far below 1 with a scale to match: their bits count like those of others (at 2^-18 most are subnormal as
    given)."""
    c = Case(fmt, 8, 2, d, 32, [200, 0, 1100], [6, 3, 1], scale=d ** -0.5 * 2.0 ** -power)
    c.q = (c.q * np.float16(2.0 ** power)).astype(np.float16)
    c.fill()
    c.check(f"{fmt} 2^{power}", *c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_different_sizes(fmt, d):
    """Small queries beside large ones of the same sequence."""
    c = Case(fmt, 8, 2, d, 32, [200, 1100], [6, 2])
    c.q = (c.q * np.float16(2.0) ** np.array([2, -4, -10, 0, -7, -13, 5, -12], np.float16)[:, None, None]).astype(np.float16)
    c.fill()
    c.check(f"{fmt} {d}", *c.run())
