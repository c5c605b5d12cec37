"""GPU tests of the choice of pages (qgemv_kv_select) where nothing but the cluster's own order keeps its blocks together: calls
without queries, whose scores are due at once, on clusters of every size.  Choices equal the definition's."""
import numpy as np
import pytest

from bit_weight_only_gb300 import build, qgemv
from test_gpu_selected_pages import batch, choice, i32

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


@pytest.mark.parametrize("hkv, d", [(1, 64), (8, 128), (40, 64)])
@pytest.mark.parametrize("entries", [200, 257, 513, 1025, 5000])
def test_sequences_without_queries(entries, hkv, d):
    """Scores of 0 for every page: the earliest ones, and those with NaN before them; beside a sequence that has a query."""
    page, n_pages = 16, 300
    c = qgemv.KVCache("int8", n_pages, page, hkv, d)
    s = qgemv.KeySummary(c)
    g = torch.Generator(device="cuda").manual_seed(entries)
    s.codes.random_(-127, 128, generator=g)
    s.scales.uniform_(0.5, 2.0, generator=g)
    s.scales[7, -1] = float("nan")
    sums, scales = s.codes.cpu().numpy().astype(np.int64), s.scales.cpu().numpy()
    rng = np.random.default_rng(hkv)
    lens, new = [entries * page - 3, entries * page // 2], [0, 1]
    table = rng.integers(0, n_pages, (2, entries)).astype(np.int32)
    q, _, cu = batch(entries, [0, 0], new, 2 * hkv, d, page, n_pages)
    for _ in range(20):
        pages, got = c.select(q, i32(table), i32(lens), i32(cu), summary=s, n_select=33)
    qh = q.cpu().numpy()
    for b in range(2):
        want, length = choice(qh[cu[b]:cu[b + 1]], 2, list(table[b]), lens[b], 33, page, sums, scales)
        assert pages[b].tolist() == want and int(got[b]) == length
    pages, got = c.select(q[:0], i32(table), i32(lens), i32([0, 0, 0]), summary=s, n_select=33)
    for b in range(2):
        want, length = choice(qh[:0], 2, list(table[b]), lens[b], 33, page, sums, scales)
        assert pages[b].tolist() == want and int(got[b]) == length
