"""Host-side checks of the rotary positions, the selection of beams, the page pool and the selection of pages (no GPU needed):
sizes, the rotary plan, and refusals before anything is launched."""
import ctypes
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

from bit_weight_only_gb300 import build, qgemv

ARG, ALIGN, OK = qgemv.QGEMV_ERR_ARG, qgemv.QGEMV_ERR_ALIGN, qgemv.QGEMV_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qgemv.load()


def cache(**kw):
    d = {"pages": 4096, "format": qgemv.KV_INT8, "head_dim": 128, "kv_heads": 2, "page_tokens": 64, "n_pages": 4, **kw}
    return ctypes.byref(qgemv.KvCacheDesc(*[d[n] for n, _ in qgemv.KvCacheDesc._fields_]))


def call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


ROWS = {"plan": 256, "pairs": 64, "pairing": 0, "axes": 1, "positions": 64, "dtype": 1, "heads": 8, "d": 128, "x": 256,
        "xt": 1024, "xh": 128, "n": 5, "out_dtype": 1, "out": 1 << 20, "ot": 1024, "oh": 128, "stream": None}
WRITE = {"cache": None, "plan": 256, "pairs": 64, "pairing": 1, "axes": 3, "positions": 64, "dtype": 1, "q": 256, "qt": 1024,
         "qh": 128, "heads": 8, "k": 256, "kt": 256, "kh": 128, "v": 256, "vt": 256, "vh": 128, "slots": 64, "n": 5,
         "out_dtype": 1, "out": 1 << 20, "ot": 1024, "oh": 128, "stream": None}
BEAM = {"dtype": 0, "logits": 256, "stride": 1000, "vocab": 1000, "scores": 256, "seqs": 2, "beams": 4, "width": 8, "os": 256,
        "ob": 256, "ot": 256, "ws": 256, "ws_bytes": 1 << 30, "stream": None}
RESERVE = {"refs": 256, "n_pages": 100, "page": 16, "table": 64, "stride": 4, "rows": 2, "have": 64, "need": 64, "missing": 64,
           "stream": None}
FORK = {"refs": 256, "n_pages": 100, "page": 16, "table": 1 << 20, "stride": 4, "rows": 2, "parents": 64, "n": 3, "lens": 64,
        "new": 2 << 20, "src": 64, "dst": 64, "tokens": 64, "missing": 64, "stream": None}
RELEASE = {"refs": 256, "n_pages": 100, "page": 16, "table": 64, "stride": 4, "rows": 2, "lens": 64, "keep": None,
           "stream": None}
COMPACT = {"refs": 256, "n_pages": 100, "table": 1 << 20, "stride": 4, "rows": 2, "new": 2 << 20, "src": 64, "dst": 64,
           "n_moves": 50, "ws": 256, "ws_bytes": 1 << 20, "stream": None}
COPY = {"cache": None, "src": 64, "dst": 64, "tokens": None, "n": 3, "stream": None}
SUMMARY = {"cache": None, "pages": 64, "n": 3, "codes": 256, "scales": 64, "stream": None}
SELECT = {"cache": None, "codes": 256, "scales": 64, "table": 64, "stride": 4, "seqs": 2, "ctx": 64, "q": 256, "qt": 1024,
          "qh": 128, "heads": 8, "cu": 64, "n": 5, "select": 3, "pages": 64, "lens": 64, "stream": None}
PAGES = {"cache": None, "pages": 64, "stride": 4, "n_seqs": 2, "ctx": 64, "q": 256, "qt": 1024, "qh": 128, "heads": 8,
         "cu": 64, "n": 5, "masks": None, "max_ctx": 100, "max_new": 3, "scale": 1.0, "out": 256, "ot": 1024, "oh": 128,
         "lse": None, "ws": 256, "ws_bytes": 1 << 40, "stream": None}


@pytest.mark.parametrize("bad, code", [({"pages": None}, ARG), ({"pages": 4100}, ALIGN), ({"format": 9}, ARG), ({"head_dim": 96}, ARG),
                                       ({"page_tokens": 24}, ARG), ({"n_pages": 0}, ARG), ({"kv_heads": 0}, ARG)])
def test_bad_caches_are_refused(lib, bad, code):
    for fn, d in ((lib.qgemv_kv_write_rotated, WRITE), (lib.qgemv_kv_copy_pages, COPY), (lib.qgemv_kv_summarize, SUMMARY),
                  (lib.qgemv_kv_select, SELECT), (lib.qgemv_attn_pages, PAGES)):
        assert call(fn, d, {"cache": cache(**bad)}) == code
        assert call(fn, d, {"cache": None}) == ARG


@pytest.mark.parametrize("kw, code", [({"plan": None}, ARG), ({"plan": 264}, ALIGN), ({"pairs": 0}, ARG), ({"pairs": 65}, ARG),
                                      ({"pairing": 2}, ARG), ({"axes": 0}, ARG), ({"axes": 5}, ARG), ({"positions": None}, ARG),
                                      ({"positions": 66}, ALIGN), ({"dtype": 3}, ARG), ({"out_dtype": 3}, ARG), ({"heads": 0}, ARG),
                                      ({"heads": 1025}, ARG), ({"n": -1}, ARG), ({"out": None}, ARG), ({"ot": 512}, ARG),
                                      ({"oh": 64}, ARG), ({"out": 264}, ALIGN), ({"n": 0}, OK)])
def test_rotations_refusals(lib, kw, code):
    assert call(lib.qgemv_rope_rows, ROWS, kw) == code
    assert call(lib.qgemv_kv_write_rotated, WRITE, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"x": None}, ARG), ({"x": 264}, ALIGN), ({"xt": 1001}, ALIGN), ({"xh": -128}, ARG),
                                      ({"d": 96}, ARG), ({"d": 64}, ARG)])
def test_rotated_rows_refusals(lib, kw, code):
    assert call(lib.qgemv_rope_rows, ROWS, kw) == code


@pytest.mark.parametrize("kw, code", [({"q": None}, ARG), ({"k": None}, ARG), ({"v": None}, ARG), ({"slots": None}, ARG),
                                      ({"slots": 68}, ALIGN), ({"k": 264}, ALIGN), ({"vt": 257}, ALIGN), ({"kh": 4}, ALIGN)])
def test_rotated_write_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_write_rotated, WRITE, {"cache": cache(), **kw}) == code


def test_the_plan_is_turns_in_fixed_point(lib):
    """round(2^64 f / 2 pi) mod 2^64, and the axis, for each pair."""
    getcontext().prec = 90
    pi = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"))
    f = np.array([1.0, 1e-4, -0.3, 1024.0, -1024.0, 1e-30, 0.0, 5e-324, 0.1234567890123, -1e-19, 10000.0 ** (-63 / 64), 6.25])
    axes = np.arange(len(f), dtype=np.int32) % 4
    plan = np.zeros((len(f), 2), dtype=np.uint64)
    qgemv.qgemv_rope_plan(f.ctypes.data, axes.ctypes.data, len(f), plan.ctypes.data)
    for x, a, (turns, axis) in zip(f, axes, plan):
        want = Fraction(float(x)) * 2 ** 64 / (2 * pi)
        off = (int(turns) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1 and axis == a
    assert qgemv.qgemv_rope_plan_bytes(64) == 1024 and qgemv.qgemv_rope_plan_bytes(0) == qgemv.qgemv_rope_plan_bytes(65) == 0
    for bad in ({0: float("nan")}, {0: float("inf")}, {0: 1025.0}):
        g = f.copy()
        g[0] = bad[0]
        assert lib.qgemv_rope_plan(g.ctypes.data, axes.ctypes.data, len(f), plan.ctypes.data) == ARG
    axes[0] = 4
    assert lib.qgemv_rope_plan(f.ctypes.data, axes.ctypes.data, len(f), plan.ctypes.data) == ARG
    assert lib.qgemv_rope_plan(None, axes.ctypes.data, len(f), plan.ctypes.data) == ARG
    assert lib.qgemv_rope_plan(f.ctypes.data, axes.ctypes.data, 65, plan.ctypes.data) == ARG


@pytest.mark.parametrize("kw, code", [({"dtype": 3}, ARG), ({"logits": None}, ARG), ({"logits": 258}, ALIGN), ({"stride": -1}, ARG),
                                      ({"vocab": 0}, ARG), ({"vocab": (1 << 30) + 1}, ARG), ({"scores": None}, ARG),
                                      ({"scores": 258}, ALIGN), ({"seqs": -1}, ARG), ({"beams": 0}, ARG), ({"beams": 65}, ARG),
                                      ({"width": 0}, ARG), ({"width": 65}, ARG), ({"os": None}, ARG), ({"ob": None}, ARG),
                                      ({"ot": None}, ARG), ({"ot": 258}, ALIGN), ({"ws": None}, ARG), ({"ws": 264}, ALIGN),
                                      ({"ws_bytes": 100}, ARG), ({"seqs": 0}, OK)])
def test_beam_refusals(lib, kw, code):
    assert call(lib.qgemv_beam_select, BEAM, kw) == code


def test_beam_workspace_sizes(lib):
    assert qgemv.qgemv_beam_ws_bytes(1, 4, 32000, 8) >= 4 * 8 * 8
    assert qgemv.qgemv_beam_ws_bytes(0, 4, 32000, 8) == qgemv.qgemv_beam_ws_bytes(1, 4, 32000, 8)
    for bad in ((-1, 4, 100, 8), (1, 0, 100, 8), (1, 65, 100, 8), (1, 4, 0, 8), (1, 4, 100, 0), (1, 4, 100, 65)):
        assert qgemv.qgemv_beam_ws_bytes(*bad) == 0


BAD_POOL = [({"refs": None}, ARG), ({"refs": 258}, ALIGN), ({"n_pages": 0}, ARG), ({"n_pages": 1 << 31}, ARG), ({"rows": -1}, ARG),
            ({"rows": 4097}, ARG), ({"stride": -1}, ARG), ({"stride": (1 << 20) + 1}, ARG), ({"table": None}, ARG)]


@pytest.mark.parametrize("kw, code", BAD_POOL)
def test_bad_pools_are_refused(lib, kw, code):
    for fn, d in ((lib.qgemv_pool_reserve, RESERVE), (lib.qgemv_pool_fork, FORK), (lib.qgemv_pool_release, RELEASE),
                  (lib.qgemv_pool_compact, COMPACT)):
        assert call(fn, d, kw) == code


@pytest.mark.parametrize("name, kw, code", [
    ("reserve", {"page": 24}, ARG), ("reserve", {"have": None}, ARG), ("reserve", {"need": None}, ARG), ("reserve", {"missing": None}, ARG),
    ("reserve", {"need": 66}, ALIGN), ("reserve", {"rows": 0}, OK), ("reserve", {"stride": 0}, OK),
    ("fork", {"page": 512}, ARG), ("fork", {"parents": None}, ARG), ("fork", {"lens": None}, ARG), ("fork", {"new": None}, ARG),
    ("fork", {"src": None}, ARG), ("fork", {"dst": None}, ARG), ("fork", {"tokens": None}, ARG), ("fork", {"missing": None}, ARG),
    ("fork", {"n": 4097}, ARG), ("fork", {"n": -1}, ARG), ("fork", {"src": 65}, ALIGN), ("fork", {"new": 1 << 20}, ARG),
    ("fork", {"new": (1 << 20) + 28}, ARG), ("fork", {"new": (1 << 20) - 44}, ARG), ("fork", {"rows": 0, "n": 0}, OK),
    ("release", {"page": 0}, ARG), ("release", {"lens": None}, ARG), ("release", {"keep": 3}, ALIGN), ("release", {"rows": 0}, OK),
    ("compact", {"new": None}, ARG), ("compact", {"src": None}, ARG), ("compact", {"n_moves": 49}, ARG), ("compact", {"n_moves": 101}, ARG),
    ("compact", {"ws": None}, ARG), ("compact", {"ws_bytes": 400}, ARG), ("compact", {"ws": 258}, ALIGN), ("compact", {"new": (1 << 20) + 4}, ARG)])
def test_pool_refusals(lib, name, kw, code):
    fn, d = {"reserve": (lib.qgemv_pool_reserve, RESERVE), "fork": (lib.qgemv_pool_fork, FORK),
             "release": (lib.qgemv_pool_release, RELEASE), "compact": (lib.qgemv_pool_compact, COMPACT)}[name]
    assert call(fn, d, kw) == code


def test_pool_workspace_sizes(lib):
    assert qgemv.qgemv_pool_ws_bytes(1) >= 4 and qgemv.qgemv_pool_ws_bytes(100000) >= 400000
    assert qgemv.qgemv_pool_ws_bytes(0) == qgemv.qgemv_pool_ws_bytes(1 << 31) == 0


@pytest.mark.parametrize("kw, code", [({"src": None}, ARG), ({"dst": None}, ARG), ({"n": -1}, ARG), ({"n": 1 << 31}, ARG),
                                      ({"src": 66}, ALIGN), ({"tokens": 66}, ALIGN), ({"n": 0}, OK)])
def test_copy_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_copy_pages, COPY, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"pages": None}, ARG), ({"pages": 66}, ALIGN), ({"n": -1}, ARG), ({"codes": None}, ARG),
                                      ({"codes": 264}, ALIGN), ({"scales": None}, ARG), ({"scales": 66}, ALIGN), ({"n": 0}, OK)])
def test_summary_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_summarize, SUMMARY, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"codes": None}, ARG), ({"scales": None}, ARG), ({"codes": 8}, ALIGN), ({"heads": 7}, ARG),
                                      ({"heads": 0}, ARG), ({"q": None}, ARG), ({"q": 264}, ALIGN), ({"qt": 1001}, ALIGN),
                                      ({"cu": None}, ARG), ({"ctx": None}, ARG), ({"table": None}, ARG), ({"pages": None}, ARG),
                                      ({"lens": None}, ARG), ({"lens": 66}, ALIGN), ({"select": -1}, ARG),
                                      ({"select": (1 << 20) + 1}, ARG), ({"stride": 49153}, ARG), ({"stride": -1}, ARG),
                                      ({"n": -1}, ARG), ({"seqs": -1}, ARG), ({"seqs": 0}, OK)])
def test_select_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_select, SELECT, {"cache": cache(), **kw}) == code


def test_select_widths(lib):
    # a context's end inside a page, and 64 drafted tokens behind it
    for page in (16, 32, 64, 128, 256):
        assert qgemv.qgemv_kv_select_width(page, 5) == 5 + -(-(page - 1 + 64) // page)
    for bad in ((24, 5), (8, 5), (64, -1), (64, (1 << 20) + 1)):
        assert qgemv.qgemv_kv_select_width(*bad) == 0


@pytest.mark.parametrize("kw, code", [({"heads": 7}, ARG), ({"q": None}, ARG), ({"out": None}, ARG), ({"ctx": None}, ARG),
                                      ({"pages": None}, ARG), ({"ot": 100}, ARG), ({"qt": 1025}, ALIGN), ({"ws": None}, ARG),
                                      ({"ws_bytes": 100}, ARG), ({"n": 0}, OK), ({"n_seqs": 0}, OK)])
def test_attend_pages_refusals(lib, kw, code):
    assert call(lib.qgemv_attn_pages, PAGES, {"cache": cache(), **kw}) == code
