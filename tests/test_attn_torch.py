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


def cache(**kw):
    return qgemv.KVCache("int8", 4, 16, 2, 64, device="cpu")


def attend(c, n=5, **kw):
    d = {"q": Stand((n, 4, 64)), "table": Stand((2, 3), torch.int32), "ctx_lens": Stand((2,), torch.int32),
         "cu_q": Stand((3,), torch.int32), "masks": Stand((n,), torch.int64), "out": Stand((n, 4, 64)),
         "lse": Stand((n, 4), torch.float32), **kw}
    ws = qgemv.AttnWorkspace.__new__(qgemv.AttnWorkspace)
    ws.nbytes, ws.ptr, ws.buffer = 1 << 20, 4096, Stand((1 << 20,), torch.uint8)
    return c.attend(d["q"], d["table"], d["ctx_lens"], d["cu_q"], d["masks"], max_ctx=9, max_new=3, workspace=ws, out=d["out"],
                    lse=d["lse"], stream=1)


@pytest.mark.parametrize("dtype", [torch.int64, torch.uint64])
@pytest.mark.parametrize("bad", [{"shape": (4,)}, {"shape": (6,)}, {"shape": (5, 1)}, {"shape": (5,), "strides": (2,)},
                                 {"shape": (5,), "device": "cpu"}])
def test_masks_of_either_type_are_checked(no_launch, dtype, bad):
    with pytest.raises(ValueError, match="masks"):
        attend(cache(), masks=Stand(**{"dtype": dtype, **bad}))


@pytest.mark.parametrize("dtype", [torch.int32, torch.float32, torch.bool])
def test_masks_of_other_types_are_refused(no_launch, dtype):
    with pytest.raises(ValueError, match="masks"):
        attend(cache(), masks=Stand((5,), dtype))


@pytest.mark.parametrize("dtype", [torch.int64, torch.uint64])
def test_right_masks_are_taken(no_launch, dtype):
    with pytest.raises(AssertionError, match="launched"):
        attend(cache(), masks=Stand((5,), dtype))
