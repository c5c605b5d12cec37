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
@pytest.mark.parametrize("new", [4, 20])
def test_a_seen_nan_counts_at_any_score(fmt, new):
    """A drafted token whose values are NaN, far below the others in score: exp is small there, but not 0."""
    c = Case(fmt, 4, 1, 128, 32, [40], [new], masks="tree")
    c.q[:] = 1
    c.k[:] = 1
    hit = 40 + 1
    c.k[hit] = -20
    c.v[hit, 0, 37] = np.nan
    c.fill()
    c.check("far NaN", *c.run())
    sees = [(m >> 1) & 1 for m in c.masks]
    assert any(sees) and not all(sees)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size", [5.25e5, 1e6, 3e38])
def test_groups_beyond_the_range_of_their_scale(kind, size):
    """Q4_0 keeps scales as fp16: a group of 32 whose scale is past them is all NaN, as one with an infinity; the groups beside
    it, and the rows that do not see it, are what they were."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[kind]
    for at in (7, 40 + 2):                                        # a cached and a drafted token
        c = Case("q4_0", 4, 1, 128, 32, [40], [9])
        c.fill()
        k, v = (torch.from_numpy(x).to(dt) for x in (c.k, c.v))
        v[at, 0, 32:64] = size * torch.linspace(-1, 1, 32)
        v[at, 0, 32] = -size
        slots = i64([int(c.table[0, at // 32]) * 32 + at % 32])
        c.cache.write(k[at:at + 1].cuda(), v[at:at + 1].cuda(), slots)
        back = c.cache.read(i32(c.table), i32([at]), i32([0, 1]), 1, dtype=torch.float32)[1][0, 0].cpu()
        assert torch.isnan(back[32:64]).all()
        c.k, c.v = c.k.astype(np.float32), c.v.astype(np.float32)
        c.k[at], c.v[at] = k[at].float().numpy(), v[at].float().numpy()
        assert np.array_equal(back[:32].numpy(), ref.quantised("q4_0", c.v[at, 0, :32]).astype(np.float32))
        c.v[at, 0, 32:64] = np.nan
        c.check("values", *c.run())
        # keys: every row that sees the token is NaN
        c = Case("q4_0", 4, 1, 128, 32, [40], [9]).fill()
        k = torch.from_numpy(c.k).to(dt)
        k[at, 0, 32:64] = size * torch.linspace(-1, 1, 32)
        k[at, 0, 32] = -size
        c.cache.write(k[at:at + 1].cuda(), torch.from_numpy(c.v[at:at + 1]).to(dt).cuda(), slots)
        out, lse = c.run()
        sees = [at < 40 or (m >> (at - 40)) & 1 for m in c.masks]
        for i, s in enumerate(sees):
            assert torch.isnan(out[i]).all() == bool(s) and torch.isnan(lse[i]).all() == bool(s), i
    # the largest group that the scale holds
    cache = qgemv.KVCache("q4_0", 1, 16, 1, 64)
    x = torch.full((1, 1, 64), 65504.0 * 8, device="cuda")
    cache.write(x, -x, i64([0]))
    k, v = cache.read(i32([[0]]), None, i32([0, 1]), 1, dtype=torch.float32)
    assert (k == 65504.0 * 8).all() and (v == -65504.0 * 8).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_different_sizes(fmt, d):
    """Small queries beside large ones of the same sequence."""
    c = Case(fmt, 8, 2, d, 32, [200, 1100], [6, 2])
    c.q = (c.q * np.float16(2.0) ** np.array([2, -4, -10, 0, -7, -13, 5, -12], np.float16)[:, None, None]).astype(np.float16)
    c.fill()
    c.check(f"{fmt} {d}", *c.run())
