"""GPU tests of the rotary positions (qgemv_rope_rows, qgemv_kv_write_rotated).

Tolerance of a rotated value a cos - b sin: the angle is a fixed-point number of turns off by |position| 2^-65 and cut to 2^-32,
then rounded to fp32 as a number of half turns of at most 1 (2^-25): pi 2^-25 + 2 pi 2^-32 radians, below 2^-23.  sincospif is
documented to within 2 units in the last place: 2^-22 for values up to 1.  The product and the sum round three times: 2^-24 each of
(|a| + |b|).  Together below (2^-23 + 2^-22 + 3 * 2^-24) (|a| + |b|) < 2^-21 (|a| + |b|); then half a step of the output's type.
"""
import numpy as np
import pytest

import attn_reference as ref
from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()


def rows(seed, kind, *shape):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32) * 3).to(TYPES[kind]).cuda()


def definition(x, positions, sections, freqs, pairs):
    """(rotated, bound without the output's rounding) in 64 bits; x [n, heads, d], positions [n, axes]."""
    x = x.detach().cpu().double().numpy()
    y, bound = x.copy(), np.zeros_like(x)
    n = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    for j in range(n):
        i, k = (j, j + n) if pairs == "halves" else (2 * j, 2 * j + 1)
        angle = positions[:, axis[j]].astype(np.float64) * freqs[j]
        far = (np.abs(angle) * 2.0 ** -52)[:, None]  # the product's own rounding here
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = x[..., i], x[..., k]
        y[..., i], y[..., k] = a * c - b * s, a * s + b * c
        bound[..., i] = bound[..., k] = (2.0 ** -21 + far) * (np.abs(a) + np.abs(b))
    return y, bound


def check(got, want, kind):
    y, bound = want
    got = got.detach().cpu().double().numpy()
    assert np.all(np.abs(got - y) <= bound + HALF[kind] * 1.001 * np.abs(y) + TINY[kind])


def places(seed, n, axes, far=1 << 20):
    g = np.random.default_rng(seed)
    return g.integers(-far, far, (n, axes)).astype(np.int32)


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("d, sections", [(128, [64]), (128, [16, 24, 24]), (128, [9, 23, 24]), (128, [1]), (128, [5, 0, 8, 2]),
                                         (64, [32]), (64, [10, 11]), (64, [8, 8]), (64, [31])])
@pytest.mark.parametrize("kind, out, heads", [("f32", "f16", 5), ("f16", "f16", 8), ("bf16", "f32", 1), ("f32", "bf16", 17)])
def test_rows(d, sections, pairs, kind, out, heads):
    n = 37
    x, pos = rows(d + heads, kind, n, heads, d), places(1, n, len(sections))
    r = qgemv.Rotary(d, sections, pairs=pairs)
    got = r.rotate(x, gpu(pos), dtype=TYPES[out])
    freqs = [10000.0 ** (-j / sum(sections)) for j in range(sum(sections))]
    check(got, definition(x, pos, sections, freqs, pairs), out)
    behind = got[..., 2 * sum(sections):]
    assert torch.equal(behind, x[..., 2 * sum(sections):].to(TYPES[out]))


@pytest.mark.parametrize("n", [0, 1, 2, 7, 300])
def test_numbers_of_tokens(n):
    x, pos = rows(n, "f32", n, 40, 128), places(n, n, 1, 100000)
    got = qgemv.Rotary(128, [64], base=500000.0).rotate(x, gpu(pos))
    assert got.shape == x.shape and got.dtype == torch.float32
    check(got, definition(x, pos, [64], [500000.0 ** (-j / 64) for j in range(64)], "halves"), "f32")


def test_far_positions_lose_nothing():
    """Positions up to the type's ends, and frequencies whose turns are exact: quarter turns come out as exchanges."""
    pos = np.array([[0], [1], [-1], [2 ** 31 - 1], [-2 ** 31], [1234567891]], np.int32)
    x = rows(3, "f32", 6, 2, 64)
    freqs = [1.0, -0.5, 2.0 ** -20, 1000.0] + [0.1] * 28
    got = qgemv.Rotary(64, [32], freqs=freqs).rotate(x, gpu(pos))
    y = x.cpu().double().numpy().copy()
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    bound = np.zeros_like(y)
    for t in range(6):
        for j, f in enumerate(freqs):
            turn = float((Decimal(int(pos[t, 0])) * Decimal(f)) % two_pi)
            a, b = x[t, :, j].cpu().double().numpy(), x[t, :, j + 32].cpu().double().numpy()
            y[t, :, j], y[t, :, j + 32] = a * np.cos(turn) - b * np.sin(turn), a * np.sin(turn) + b * np.cos(turn)
            bound[t, :, j] = bound[t, :, j + 32] = 2.0 ** -21 * (np.abs(a) + np.abs(b))
    check(got, (y, bound), "f32")


def test_strides_and_in_place():
    """Slices of a stacked product, token-major and head-major, and rows turned where they are."""
    r = qgemv.Rotary(128, [20, 20, 16])
    pos = gpu(places(4, 50, 3))
    stack = rows(5, "f16", 50, 12, 128)
    want = r.rotate(stack[:, 2:9].contiguous(), pos)
    assert torch.equal(r.rotate(stack[:, 2:9], pos), want)
    by_head = stack[:, 2:9].permute(1, 0, 2).contiguous().permute(1, 0, 2)
    assert torch.equal(r.rotate(by_head, pos), want)
    out = torch.full((50, 9, 128), 7.0, dtype=torch.float16, device="cuda")
    assert r.rotate(stack[:, 2:9], pos, out=out[:, 1:8]).data_ptr() == out[:, 1:8].data_ptr()
    assert torch.equal(out[:, 1:8], want) and bool((out[:, 0] == 7).all()) and bool((out[:, 8] == 7).all())
    for pairs, sections in (("halves", [20, 20, 16]), ("halves", [9, 20, 20]), ("neighbours", [9, 20, 20])):
        r = qgemv.Rotary(128, sections, pairs=pairs)
        kept = stack.clone()
        want = r.rotate(kept[:, 2:9], pos)
        r.rotate(kept[:, 2:9], pos, out=kept[:, 2:9])
        assert torch.equal(kept[:, 2:9], want) and torch.equal(kept[:, :2], stack[:, :2]) and torch.equal(kept[:, 9:], stack[:, 9:])


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_backwards(pairs):
    """Negative positions undo a rotation, and give its gradient: that of the formula, and differences'."""
    sections, d = [12, 20], 64
    r = qgemv.Rotary(d, sections, pairs=pairs)
    x, pos = rows(6, "f32", 9, 3, d), places(6, 9, 2, 5000)
    back = r.rotate(r.rotate(x, gpu(pos)), gpu(-pos))
    big = float(x.abs().max())
    assert float((back - x).abs().max()) <= 2 * 2 * 2.0 ** -21 * 2 * big  # twice the bound of values up to 2 |x|
    g = rows(7, "f32", 9, 3, d)
    grad = r.rotate(g, gpu(-pos))
    freqs = [10000.0 ** (-j / 32) for j in range(32)]
    # of the formula: x enters as a cos - b sin, a sin + b cos
    leaf = x.cpu().double().requires_grad_()
    axis = np.repeat(np.arange(2), sections)
    angle = torch.from_numpy(pos[:, axis].astype(np.float64) * np.array(freqs))[:, None]
    a, b = (leaf[..., :32], leaf[..., 32:]) if pairs == "halves" else (leaf[..., 0::2], leaf[..., 1::2])
    y = torch.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()])
    gg = g.cpu().double()
    want = torch.stack([gg[..., :32], gg[..., 32:]] if pairs == "halves" else [gg[..., 0::2], gg[..., 1::2]])
    (y * want).sum().backward()
    assert float((grad.cpu().double() - leaf.grad).abs().max()) <= 2.0 ** -20 * 2 * float(g.abs().max())
    # differences: a rotation is linear, so one step is the derivative up to the two results' bounds
    e = rows(8, "f32", 9, 3, d)
    slope = ((r.rotate(x + e, gpu(pos)) - r.rotate(x, gpu(pos))).double() * g.double()).sum()
    off = 9 * 3 * d * float(g.abs().max()) * 2.0 ** -20 * 2 * 2 * (big + float(e.abs().max()))
    assert abs(float(slope) - float((grad.double() * ((x + e).double() - x.double())).sum())) <= off


def test_infinities_stay_with_their_pair():
    for pairs in ("halves", "neighbours"):
        for n in (24, 21):
            x = rows(9, "f32", 4, 2, 64)
            x[0, 0, 3] = float("nan")
            x[1, 1, 60] = float("inf")     # behind the pairs
            x[2, 0, 5] = float("inf")
            got = qgemv.Rotary(64, [n], pairs=pairs).rotate(x, gpu(places(9, 4, 1)))
            touched = {(0, 0, 3), (2, 0, 5)} | ({(0, 0, 3 + n), (2, 0, 5 + n)} if pairs == "halves" else {(0, 0, 2), (2, 0, 4)})
            wrong = {tuple(i) for i in np.argwhere(~np.isfinite(got.cpu().numpy()))}
            assert wrong - {(1, 1, 60)} <= touched and (0, 0, 3) in wrong and float(got[1, 1, 60]) == float("inf")


@pytest.mark.parametrize("fmt", ["f16", "int8", "q4_0"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d, hq, hkv, sections, pairs", [(128, 40, 8, [64], "halves"), (128, 7, 7, [9, 23, 24], "halves"),
                                                         (64, 16, 2, [28], "neighbours"), (64, 3, 1, [9, 8], "halves")])
def test_rotated_write(fmt, kind, d, hq, hkv, sections, pairs):
    """The cache holds what write() makes of the rotated fp32 keys, and of v as it is; q is rotate()'s; skipped slots change
    nothing and their tokens' q is there."""
    n, page, n_pages = 75, 32, 4
    stack = rows(d + hq, kind, n, hq + 2 * hkv, d)
    q, k, v = stack[:, :hq], stack[:, hq:hq + hkv], stack[:, hq + hkv:]
    pos = gpu(places(2, n, len(sections)))
    slots = np.random.default_rng(3).permutation(n_pages * page)[:n].astype(np.int64)
    slots[[3, 40]] = -1, n_pages * page
    r = qgemv.Rotary(d, sections, pairs=pairs)
    a, b = (qgemv.KVCache(fmt, n_pages, page, hkv, d) for _ in range(2))
    a.pages.fill_(0x3C)
    b.pages.fill_(0x3C)
    got = a.write_rotated(r, q, k, v, pos, gpu(slots))
    b.write(r.rotate(k, pos, dtype=torch.float32), v.float(), gpu(slots))
    assert torch.equal(a.pages, b.pages)
    assert got.dtype == torch.float16 and torch.equal(got, r.rotate(q, pos, dtype=torch.float16))
    for out in (torch.bfloat16, torch.float32):
        wide = torch.empty(n, hq + 1, d, dtype=out, device="cuda")[:, 1:]
        a.write_rotated(r, q, k, v, pos, gpu(slots), out=wide)
        assert torch.equal(wide, r.rotate(q, pos, dtype=out))
    # and against the definition: fp16 keys are the rotated values, rounded
    if fmt == "f16":
        here = np.flatnonzero((slots >= 0) & (slots < n_pages * page))
        table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
        back, _ = a.read(table, None, torch.tensor([0, n_pages * page], dtype=torch.int32, device="cuda"), n_pages * page, dtype=torch.float32)
        freqs = [10000.0 ** (-j / sum(sections)) for j in range(sum(sections))]
        check(back[gpu(slots[here])], definition(k[gpu(here)], pos.cpu().numpy()[here], sections, freqs, pairs), "f16")


def test_codes_are_the_quantiser_of_the_rotated_keys():
    n, h, d = 40, 2, 128
    k = rows(11, "f32", n, h, d)
    pos = gpu(places(11, n, 1))
    r = qgemv.Rotary(d, [64])
    turned = r.rotate(k, pos).cpu().numpy()
    for fmt in ("int8", "q4_0"):
        c = qgemv.KVCache(fmt, 3, 16, h, d)
        c.write_rotated(r, k, k, k, pos, torch.arange(n, device="cuda"))
        got, _ = c.read(torch.arange(3, dtype=torch.int32, device="cuda")[None], None, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, dtype=torch.float32)
        assert np.array_equal(got.cpu().numpy(), ref.quantised(fmt, turned).astype(np.float32))


def test_streams_and_graphs():
    """On a stream of its own, and captured and replayed with other rows and positions."""
    r = qgemv.Rotary(128, [16, 24, 24])
    c = qgemv.KVCache("int8", 4, 16, 2, 128)
    x, y = rows(12, "f16", 30, 8, 128), rows(13, "f16", 30, 8, 128)
    pos, pos2 = gpu(places(12, 30, 3)), gpu(places(13, 30, 3))
    slots = torch.arange(30, device="cuda")

    def step(x, pos, **kw):
        return c.write_rotated(r, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, **kw)
    want, pages = step(x, pos), c.pages.clone()
    want2, pages2 = step(y, pos2), c.pages.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(x, pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(c.pages, pages)
    xs, ps = x.clone(), pos.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(xs, ps)
    xs.copy_(y)
    ps.copy_(pos2)
    g.replay()
    assert torch.equal(got, want2) and torch.equal(c.pages, pages2)
    xs.copy_(x)
    ps.copy_(pos)
    g.replay()
    assert torch.equal(got, want) and torch.equal(c.pages, pages)
