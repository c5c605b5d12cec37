"""Checks of arguments in the torch-level calls of rotary positions, beams, the page pool and selected pages, before anything is
launched (no GPU needed)."""
import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
from test_attn_torch import Stand, on, ws  # noqa: E402

F16, F32, I32, I64 = torch.float16, torch.float32, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    qgemv.load()


@pytest.fixture
def launched(monkeypatch):
    """Records the device that each call is made on instead of making it; the current one is cuda:0."""
    got = []
    monkeypatch.setattr(qgemv, "_call", lambda dev, fn, *args: got.append(dev))
    return got


def rotary(device="cuda:1", head_dim=64):
    r = qgemv.Rotary.__new__(qgemv.Rotary)
    r.head_dim, r.pairs, r.axes, r.pairing, r.ptr, r._dev = head_dim, 32, 3, 0, 4096, torch.device(device).index
    return r


def pool(device="cuda:1"):
    p = qgemv.PagePool.__new__(qgemv.PagePool)
    p.n_pages, p.page_tokens, p._nbytes, p._dev = 9, 16, 4096, torch.device(device).index
    p.refs = p._state = p._ws = Stand((9,), I32, device=device)
    return p


def summary(cache):
    s = qgemv.KeySummary.__new__(qgemv.KeySummary)
    s.cache, s.codes, s.scales = cache, Stand((4, 2, 2, 64), torch.int8), Stand((4, 2), F32)
    return s


def make(call, **kw):
    """The call, on stand-ins of one device but for those in kw (name = device, or a stand-in)."""
    def t(name, shape, kind):
        other = kw.get(name)
        return other if isinstance(other, Stand) else Stand(shape, kind, device=other or "cuda:1")
    if call == "rotate":
        return rotary().rotate(t("x", (5, 4, 64), F16), t("positions", (5, 3), I32), out=t("out", (5, 4, 64), F16), stream=1)
    if call == "write_rotated":
        return on(1).write_rotated(rotary(kw.get("rotary", "cuda:1"), kw.get("head_dim", 64)), t("q", (5, 4, 64), F16), t("k", (5, 2, 64), F16),
                                   t("v", (5, 2, 64), F16), t("positions", (5, 3), I32), t("slots", (5,), I64),
                                   out=t("out", (5, 4, 64), F16), stream=1)
    if call == "beam_select":
        w = qgemv.BeamWorkspace.__new__(qgemv.BeamWorkspace)
        w.nbytes, w.ptr, w._dev = 1 << 20, 4096, torch.device(kw.get("workspace", "cuda:1")).index
        return qgemv.beam_select(t("logits", (6, 100), F32), t("scores", (2, 3), F32), 4, workspace=w, stream=1,
                                 out=(t("out0", (2, 4), F32), t("out1", (2, 4), I32), t("out2", (2, 4), I32)))
    if call == "reserve":
        return pool().reserve(t("table", (2, 3), I32), t("have", (2,), I32), t("need", (2,), I32), stream=1)
    if call == "release":
        return pool().release(t("table", (2, 3), I32), t("lens", (2,), I32), t("keep", (2,), I32), stream=1)
    if call == "copy_pages":
        return on(1).copy_pages(t("src", (3,), I32), t("dst", (3,), I32), t("tokens", (3,), I32), stream=1)
    c = on(1)
    if call == "update":
        s = summary(c)
        return s.update(t("pages", (3,), I32), stream=1)
    if call == "select":
        return c.select(t("q", (5, 4, 64), F16), t("table", (2, 3), I32), t("ctx_lens", (2,), I32), t("cu_q", (3,), I32), stream=1,
                        summary=summary(kw.get("cache", c)), n_select=kw.get("n_select", 2),
                        out=(t("pages", (2, 2, 2 + 5), I32), t("lens", (2,), I32)))
    assert call == "attend_pages"
    return c.attend_pages(t("q", (5, 4, 64), F16), t("pages", (2, 2, 7), I32), t("lens", (2,), I32), t("cu_q", (3,), I32),
                          t("masks", (5,), I64), max_ctx=9, max_new=3, workspace=ws(kw.get("workspace", "cuda:1")),
                          out=t("out", (5, 4, 64), F16), lse=t("lse", (5, 4), F32), stream=1)


NAMES = {"rotate": ["x", "positions", "out"], "write_rotated": ["rotary", "q", "k", "v", "positions", "slots", "out"],
         "beam_select": ["logits", "scores", "workspace", "out0", "out1", "out2"], "reserve": ["table", "have", "need"],
         "release": ["table", "lens", "keep"], "copy_pages": ["src", "dst", "tokens"], "update": ["pages"],
         "select": ["q", "table", "ctx_lens", "cu_q", "pages", "lens"],
         "attend_pages": ["q", "pages", "lens", "cu_q", "masks", "workspace", "out", "lse"]}


@pytest.mark.parametrize("call", list(NAMES))
def test_calls_run_on_the_device_of_their_tensors(launched, call):
    make(call)
    assert launched == [1]


@pytest.mark.parametrize("call, name", [(c, n) for c in NAMES for n in NAMES[c]])
@pytest.mark.parametrize("other", ["cuda:0", "cpu"])
def test_tensors_of_other_devices_are_refused(launched, call, name, other):
    if other == "cpu" and name in ("rotary", "workspace"):
        pytest.skip("is never on the host")
    with pytest.raises(ValueError):
        make(call, **{name: other})
    assert not launched


C1 = "cuda:1"


@pytest.mark.parametrize("call, bad", [
    ("rotate", {"x": Stand((5, 4, 128), F16, device=C1)}), ("rotate", {"positions": Stand((5, 2), I32, device=C1)}),
    ("rotate", {"positions": Stand((5, 3), I64, device=C1)}), ("rotate", {"x": Stand((5, 4, 64), torch.int8, device=C1)}),
    ("rotate", {"out": Stand((5, 3, 64), F16, device=C1)}), ("rotate", {"x": Stand((5, 4, 64), F16, (256, 64, 2), C1)}),
    ("write_rotated", {"head_dim": 128}), ("write_rotated", {"k": Stand((5, 2, 64), F32, device=C1)}),
    ("write_rotated", {"v": Stand((4, 2, 64), F16, device=C1)}), ("write_rotated", {"slots": Stand((4,), I64, device=C1)}),
    ("write_rotated", {"k": Stand((5, 3, 64), F16, device=C1)}),
    ("beam_select", {"logits": Stand((5, 100), F32, device=C1)}), ("beam_select", {"logits": Stand((6, 100), F32, (100, 2), C1)}),
    ("beam_select", {"scores": Stand((2, 3), F16, device=C1)}), ("beam_select", {"out1": Stand((2, 4), I64, device=C1)}),
    ("beam_select", {"logits": Stand((6, 100), I32, device=C1)}),
    ("reserve", {"have": Stand((3,), I32, device=C1)}), ("reserve", {"table": Stand((2, 3), I64, device=C1)}),
    ("reserve", {"table": Stand((2, 3), I32, (4, 1), C1)}), ("release", {"keep": Stand((2,), I64, device=C1)}),
    ("copy_pages", {"dst": Stand((2,), I32, device=C1)}), ("copy_pages", {"tokens": Stand((3,), I64, device=C1)}),
    ("update", {"pages": Stand((3,), I64, device=C1)}),
    ("select", {"q": Stand((5, 4, 64), F32, device=C1)}), ("select", {"pages": Stand((2, 2, 6), I32, device=C1)}),
    ("select", {"cache": None}), ("select", {"q": Stand((5, 4, 128), F16, device=C1)}),
    ("attend_pages", {"pages": Stand((2, 1, 7), I32, device=C1)}), ("attend_pages", {"q": Stand((5, 4, 64), F32, device=C1)}),
    ("attend_pages", {"lens": Stand((3,), I32, device=C1)})])
def test_wrong_tensors_are_refused(launched, call, bad):
    with pytest.raises(ValueError):
        make(call, **bad)
    assert not launched


def test_wrong_numbers_are_refused(launched):
    with pytest.raises(qgemv.QgemvError):
        make("select", n_select=-1)
    for args in ((96, [8]), (64, [33]), (64, []), (64, [8, 8, 8, 4, 4]), (64, [0]), (64, [40, -8])):
        with pytest.raises(qgemv.QgemvError):
            qgemv.Rotary(*args, device="cuda:1")
    with pytest.raises(qgemv.QgemvError):
        qgemv.Rotary(64, [32], pairs="thirds")
    with pytest.raises(qgemv.QgemvError):
        qgemv.Rotary(64, [32], freqs=[1.0] * 31)
    with pytest.raises(qgemv.QgemvError):
        qgemv.Rotary(64, [1], freqs=[float("nan")])
    for args in ((1, 65, 100, 4), (1, 4, 0, 4), (1, 4, 100, 65)):
        with pytest.raises(qgemv.QgemvError):
            qgemv.BeamWorkspace(*args)
    for args in ((0, 16), (9, 24)):
        with pytest.raises(qgemv.QgemvError):
            qgemv.PagePool(*args)
    for make_one in (lambda: qgemv.Rotary(64, [32], device="cpu"), lambda: qgemv.BeamWorkspace(1, 4, 100, 4, device="cpu"),
                     lambda: qgemv.PagePool(9, 16, device="cpu")):
        with pytest.raises(ValueError, match="CUDA"):
            make_one()
