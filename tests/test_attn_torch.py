"""Checks of arguments in the torch-level cache and attention calls, before anything is launched (no GPU needed)."""
import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    qgemv.load()


class Stand:
    """What the checks look at of a CUDA tensor."""

    def __init__(self, shape, dtype=torch.float16, strides=None, device="cuda:0"):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self._strides = torch.empty(shape, device="meta").stride() if strides is None else strides

    is_cuda = property(lambda self: self.device.type == "cuda")
    ndim = property(lambda self: len(self.shape))

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def stride(self):
        return self._strides

    def is_contiguous(self):
        return self._strides == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 4096


@pytest.fixture
def no_launch(monkeypatch):
    """The library's calls that launch kernels: the test fails where one is reached with arguments that are wrong."""
    def reached(*args):
        raise AssertionError("launched")
    monkeypatch.setattr(qgemv, "_call", reached)


def on(device):
    """A cache on a device that need not exist."""
    real = torch.empty
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                  real(shape, device=device) if device == "meta" else Stand((shape,), dtype, (1,), device))
        return qgemv.KVCache("int8", 4, 16, 2, 64, device=f"cuda:{device}")


def ws(device="cuda:0"):
    w = qgemv.AttnWorkspace.__new__(qgemv.AttnWorkspace)
    w.nbytes, w.ptr, w.buffer = 1 << 20, 4096, Stand((1 << 20,), torch.uint8, device=device)
    w._dev = w.buffer.get_device()
    return w


def attend(c, n=5, **kw):
    d = {"q": Stand((n, 4, 64)), "table": Stand((2, 3), torch.int32), "ctx_lens": Stand((2,), torch.int32),
         "cu_q": Stand((3,), torch.int32), "masks": Stand((n,), torch.int64), "out": Stand((n, 4, 64)),
         "lse": Stand((n, 4), torch.float32), **kw}
    return c.attend(d["q"], d["table"], d["ctx_lens"], d["cu_q"], d["masks"], max_ctx=9, max_new=3, workspace=ws(),
                    out=d["out"], lse=d["lse"], stream=1)


@pytest.mark.parametrize("dtype", [torch.int64, torch.uint64])
@pytest.mark.parametrize("bad", [{"shape": (4,)}, {"shape": (6,)}, {"shape": (5, 1)}, {"shape": (5,), "strides": (2,)},
                                 {"shape": (5,), "device": "cpu"}])
def test_masks_of_either_type_are_checked(no_launch, dtype, bad):
    with pytest.raises(ValueError, match="masks"):
        attend(on(0), masks=Stand(**{"dtype": dtype, **bad}))


@pytest.mark.parametrize("dtype", [torch.int32, torch.float32, torch.bool])
def test_masks_of_other_types_are_refused(no_launch, dtype):
    with pytest.raises(ValueError, match="masks"):
        attend(on(0), masks=Stand((5,), dtype))


@pytest.mark.parametrize("dtype", [torch.int64, torch.uint64])
def test_right_masks_are_taken(no_launch, dtype):
    with pytest.raises(AssertionError, match="launched"):
        attend(on(0), masks=Stand((5,), dtype))


@pytest.fixture
def launched(monkeypatch):
    """Records the device that each call is made on instead of making it; the current one is cuda:0."""
    got = []
    monkeypatch.setattr(qgemv, "_call", lambda dev, fn, *args: got.append(dev))
    return got


def arguments(call, device="cuda:1", **kw):
    """The call's arguments, stand-ins on one device, but for those in kw (name=device)."""
    at = lambda name: kw.get(name, device)  # noqa: E731
    rows = lambda name, h, kind=torch.float16: Stand((5, h, 64), kind, device=at(name))  # noqa: E731
    ints = lambda name, *shape: Stand(shape, torch.int64 if name in ("slots", "masks") else torch.int32, device=at(name))  # noqa: E731
    if call == "write":
        return (rows("k", 2), rows("v", 2), ints("slots", 5)), {}
    if call == "read":
        return (ints("table", 2, 3), ints("starts", 2), ints("cu", 3), 5), {"out": (rows("k", 2), rows("v", 2))}
    lse = Stand((5, 4), torch.float32, device=at("lse"))
    if call == "attend":
        return ((rows("q", 4), ints("table", 2, 3), ints("ctx_lens", 2), ints("cu_q", 3), ints("masks", 5)),
                {"max_ctx": 9, "max_new": 3, "workspace": ws(at("workspace")), "out": rows("out", 4), "lse": lse})
    return ((rows("q", 4), rows("k", 2), rows("v", 2), ints("cu_q", 3), ints("cu_k", 3)),
            {"max_q": 3, "workspace": ws(at("workspace")), "out": rows("out", 4), "lse": lse})


NAMES = {"write": ["k", "v", "slots"], "read": ["table", "starts", "cu", "k", "v"],
         "attend": ["q", "table", "ctx_lens", "cu_q", "masks", "workspace", "out", "lse"],
         "attn_prompt": ["q", "k", "v", "cu_q", "cu_k", "workspace", "out", "lse"]}


@pytest.mark.parametrize("call", list(NAMES))
def test_calls_run_on_the_device_of_their_tensors(launched, call):
    fn = qgemv.attn_prompt if call == "attn_prompt" else getattr(on(1), call)
    args, kw = arguments(call)
    fn(*args, **kw, stream=1)
    assert launched == [1]


@pytest.mark.parametrize("call, name", [(c, n) for c in NAMES for n in NAMES[c]])
@pytest.mark.parametrize("other", ["cuda:0", "cpu"])
def test_tensors_of_other_devices_are_refused(launched, call, name, other):
    fn = qgemv.attn_prompt if call == "attn_prompt" else getattr(on(1), call)
    args, kw = arguments(call, **{name: other})
    with pytest.raises(ValueError):
        fn(*args, **kw, stream=1)
    assert not launched


def test_caches_and_workspaces_are_not_on_the_host():
    with pytest.raises(ValueError, match="CUDA"):
        qgemv.KVCache("int8", 4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        qgemv.AttnWorkspace(1, 8, 64, device="cpu")


def test_the_device_is_current_during_a_call(monkeypatch):
    """_call makes the device current for the library and restores the one before, also when the call fails."""
    seen, now = [], [0]

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now[0] = now[0], self.dev

        def __exit__(self, *exc):
            now[0] = self.before

    monkeypatch.setattr(qgemv, "_device_now", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for dev in (0, 1):
        qgemv._call(dev, lambda *a: seen.append((now[0], a)) or 0, 5, 6)
    assert seen == [(0, (5, 6)), (1, (5, 6))] and now == [0]
    with pytest.raises(qgemv.QgemvError):
        qgemv._call(1, lambda: 1)
    assert now == [0]
