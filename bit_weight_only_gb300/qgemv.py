"""Thin ctypes binding of the C ABI in ``include/qgemv.h``.

The functions keep the C names and only marshal arguments (pointers and
sizes); every step of the computation runs in ``libqgemv.so``.  The library
is loaded on first use from ``bit_weight_only_gb300/_build``; if it is
missing, ``load()`` raises: there is no CPU fallback.

``QGemv`` wraps one handle for torch users: it takes canonical inputs as
torch tensors or numpy arrays (host or CUDA) and runs on CUDA tensors.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

Q4_0, CBK4, CBK8, PQ2_0, AQLM_2X8, AQLM_1X16, CBK4_ROW, CBK8_ROW = 1, 2, 3, 4, 5, 7, 8, 9
FORMATS = {"q4_0": Q4_0, "cbk4": CBK4, "cbk8": CBK8, "pq2_0": PQ2_0, "aqlm_2x8": AQLM_2X8,
           "aqlm_1x16": AQLM_1X16, "cbk4_row": CBK4_ROW, "cbk8_row": CBK8_ROW}
QGEMV_OK, QGEMV_ERR_ARG, QGEMV_ERR_ALIGN, QGEMV_ERR_CUDA, QGEMV_ERR_TIMEOUT, QGEMV_ERR_NOMEM = range(6)

KV_F16, KV_INT8, KV_Q4_0 = 1, 2, 3
KV_FORMATS = {"f16": KV_F16, "int8": KV_INT8, "q4_0": KV_Q4_0}
DT_F32, DT_F16, DT_BF16 = 0, 1, 2


class KvCacheDesc(ctypes.Structure):
    """``qgemv_kv_cache`` of include/qgemv.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("format", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("page_tokens", ctypes.c_int), ("n_pages", ctypes.c_int64)]


LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libqgemv.so")

_P, _I, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float

# Every exported symbol of include/qgemv.h with its ctypes signature.
_SIGNATURES = {
    "qgemv_packed_bytes": (ctypes.c_int64, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64]),
    "qgemv_create": (ctypes.c_void_p, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_create_stacked": (ctypes.c_void_p, [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64),
                                               ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "qgemv_run": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_run_residual": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_set_batch_invariant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "qgemv_set_x_int8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "qgemv_create_glu": (ctypes.c_void_p, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_xq_bytes": (ctypes.c_int64, [ctypes.c_int, ctypes.c_int64]),
    "qgemv_prepare_x_int8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_run_xq": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_quantize_x_int8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_dequant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_quantize_q4_0": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_void_p]),
    "qgemv_status": (ctypes.c_int, [ctypes.c_void_p]),
    "qgemv_run_q4_0_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                              ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "qgemv_stream_k_plan": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int,
                                           ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]),
    "qgemv_destroy": (None, [ctypes.c_void_p]),
    "qgemv_kv_bytes": (_L, [_I, _L, _I, _I, _I]),
    "qgemv_kv_write": (_I, [_P, _I, _P, _L, _L, _P, _L, _L, _P, _L, _P]),
    "qgemv_kv_read": (_I, [_P, _P, _L, _L, _P, _P, _L, _I, _P, _L, _L, _P, _L, _L, _P]),
    "qgemv_attn_ws_bytes": (_L, [_L, _I, _I]),
    "qgemv_attn_ws_init": (_I, [_P, _L, _P]),
    "qgemv_attn_status": (_I, [_P]),
    "qgemv_attn_tree": (_I, [_P, _P, _L, _L, _P, _P, _L, _L, _I, _P, _L, _P, _L, _L, _F, _P, _L, _L, _P, _P, _L, _P]),
    "qgemv_attn_prompt": (_I, [_I, _I, _I, _I, _P, _L, _L, _P, _L, _L, _P, _L, _L, _L, _P, _P, _L, _L, _L, _F,
                               _P, _L, _L, _P, _P, _L, _P]),
    "qgemv_last_error": (ctypes.c_char_p, []),
    "qgemv_last_error_code": (ctypes.c_int, []),
}

_lib = None


class QgemvError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"qgemv error {code}: {msg}")
        self.code = code


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libqgemv.so (once) and declare the ABI's signatures."""
    global _lib
    if _lib is None:
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise ImportError(f"libqgemv.so not built ({path}); run "
                              "`python -m bit_weight_only_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _kv_fmt(fmt) -> int:
    return KV_FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _check(rc: int):
    if rc != QGEMV_OK:
        raise QgemvError(rc, qgemv_last_error())
    return rc


def _stream_ptr(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream  # torch.cuda.Stream


# --------------------------------------------------------- C-ABI mirrors ----

def qgemv_packed_bytes(fmt, N: int, K: int) -> int:
    return int(load().qgemv_packed_bytes(_fmt(fmt), N, K))


def qgemv_create(fmt, N: int, K: int, packed: int, scales: int | None,
                 codebooks: int | None) -> int:
    """Pointers are raw addresses (host or device).  Returns the handle."""
    h = load().qgemv_create(_fmt(fmt), N, K, packed, scales, codebooks)
    if not h:
        raise QgemvError(qgemv_last_error_code(), qgemv_last_error())
    return h


def qgemv_create_stacked(fmt, seg_rows, K: int, packed: int, scales: int | None,
                         codebooks: int | None) -> int:
    """Several projections sharing K, rows stacked; one codebook per segment."""
    rows = (ctypes.c_int64 * len(seg_rows))(*[int(r) for r in seg_rows])
    h = load().qgemv_create_stacked(_fmt(fmt), len(seg_rows), rows, K, packed, scales, codebooks)
    if not h:
        raise QgemvError(qgemv_last_error_code(), qgemv_last_error())
    return h


def qgemv_create_glu(fmt, N: int, K: int, packed_gate: int, packed_up: int,
                     codebooks_gate: int | None = None, codebooks_up: int | None = None) -> int:
    """Gate and up projections in one handle whose runs store SiLU(gate) * up."""
    h = load().qgemv_create_glu(_fmt(fmt), N, K, packed_gate, packed_up, codebooks_gate, codebooks_up)
    if not h:
        raise QgemvError(qgemv_last_error_code(), qgemv_last_error())
    return h


def qgemv_run(h: int, x: int, M: int, y: int, stream=None) -> int:
    return _check(load().qgemv_run(h, x, M, y, _stream_ptr(stream)))


def qgemv_run_residual(h: int, x: int, M: int, y: int, residual: int, stream=None) -> int:
    return _check(load().qgemv_run_residual(h, x, M, y, residual, _stream_ptr(stream)))


def qgemv_dequant(h: int, w_out: int, stream=None) -> int:
    return _check(load().qgemv_dequant(h, w_out, _stream_ptr(stream)))


def qgemv_quantize_q4_0(w: int, N: int, K: int, packed_out: int, stream=None) -> int:
    return _check(load().qgemv_quantize_q4_0(w, N, K, packed_out, _stream_ptr(stream)))


def qgemv_run_q4_0_noalloc(packed: int, N: int, K: int, x: int, M: int, y: int,
                           stream=None) -> int:
    """Allocation-free Q4_0 GEMV on canonical device blocks (no handle)."""
    return _check(load().qgemv_run_q4_0_noalloc(packed, N, K, x, M, y, _stream_ptr(stream)))


def qgemv_set_batch_invariant(h: int, on: bool) -> int:
    return _check(load().qgemv_set_batch_invariant(h, 1 if on else 0))


def qgemv_set_x_int8(h: int, on: bool) -> int:
    return _check(load().qgemv_set_x_int8(h, 1 if on else 0))


def qgemv_quantize_x_int8(x: int, M: int, K: int, q_out: int, a_out: int, stream=None) -> int:
    return _check(load().qgemv_quantize_x_int8(x, M, K, q_out, a_out, _stream_ptr(stream)))


def qgemv_xq_bytes(M: int, K: int) -> int:
    return int(load().qgemv_xq_bytes(M, K))


def qgemv_prepare_x_int8(x: int, M: int, K: int, signs: int | None, hadamard_block: int, xq: int,
                         stream=None) -> int:
    return _check(load().qgemv_prepare_x_int8(x, M, K, signs, hadamard_block, xq, _stream_ptr(stream)))


def qgemv_run_xq(h: int, xq: int, M: int, y: int, residual: int | None = None, stream=None) -> int:
    return _check(load().qgemv_run_xq(h, xq, M, y, residual, _stream_ptr(stream)))


def qgemv_status(h: int) -> int:
    return _check(load().qgemv_status(h))


def qgemv_stream_k_plan(units: int, grid: int, units_per_row_tile: int, rows: int, split_unit: int = 1) -> list:
    """The stream-K split the handles use (host only): per CTA a dict of its
    two shared-row-tile segments, each field a pair (first, last row tile);
    "side1" and "fin" are the two flag bits."""
    out = (ctypes.c_int64 * (12 * grid))()
    _check(load().qgemv_stream_k_plan(units, grid, units_per_row_tile, rows, split_unit, out))
    keys = ("rt", "cf", "S", "r0", "nr", "flags")
    plan = [{k: (out[12 * c + 2 * i], out[12 * c + 2 * i + 1]) for i, k in enumerate(keys)}
            for c in range(grid)]
    for d in plan:
        f = d.pop("flags")
        d["side1"] = (f[0] & 1, f[1] & 1)
        d["fin"] = ((f[0] >> 1) & 1, (f[1] >> 1) & 1)
    return plan


def qgemv_destroy(h: int) -> None:
    load().qgemv_destroy(h)


def qgemv_last_error() -> str:
    return (load().qgemv_last_error() or b"").decode()


def qgemv_last_error_code() -> int:
    return int(load().qgemv_last_error_code())


def qgemv_kv_bytes(fmt, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int) -> int:
    return int(load().qgemv_kv_bytes(_kv_fmt(fmt), n_pages, page_tokens, kv_heads, head_dim))


def qgemv_kv_write(cache: KvCacheDesc, dtype: int, k: int, k_token_stride: int, k_head_stride: int, v: int,
                   v_token_stride: int, v_head_stride: int, slots: int, n_tokens: int, stream=None) -> int:
    return _check(load().qgemv_kv_write(ctypes.byref(cache), dtype, k, k_token_stride, k_head_stride, v, v_token_stride,
                                        v_head_stride, slots, n_tokens, _stream_ptr(stream)))


def qgemv_kv_read(cache: KvCacheDesc, table: int, table_stride: int, n_seqs: int, starts: int | None, cu: int,
                  n_tokens: int, dtype: int, k: int, k_token_stride: int, k_head_stride: int, v: int,
                  v_token_stride: int, v_head_stride: int, stream=None) -> int:
    return _check(load().qgemv_kv_read(ctypes.byref(cache), table, table_stride, n_seqs, starts, cu, n_tokens, dtype,
                                       k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
                                       _stream_ptr(stream)))


def qgemv_attn_ws_bytes(n_seqs: int, q_heads: int, head_dim: int) -> int:
    return int(load().qgemv_attn_ws_bytes(n_seqs, q_heads, head_dim))


def qgemv_attn_ws_init(ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_attn_ws_init(ws, ws_bytes, _stream_ptr(stream)))


def qgemv_attn_status(ws: int) -> int:
    return _check(load().qgemv_attn_status(ws))


def qgemv_attn_tree(cache: KvCacheDesc, table: int, table_stride: int, n_seqs: int, ctx_lens: int, q: int,
                    q_token_stride: int, q_head_stride: int, q_heads: int, cu_q: int, n_q: int, masks: int | None,
                    max_ctx: int, max_new: int, scale: float, out: int, out_token_stride: int, out_head_stride: int,
                    lse: int | None, ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_attn_tree(ctypes.byref(cache), table, table_stride, n_seqs, ctx_lens, q, q_token_stride,
                                         q_head_stride, q_heads, cu_q, n_q, masks, max_ctx, max_new, scale, out,
                                         out_token_stride, out_head_stride, lse, ws, ws_bytes, _stream_ptr(stream)))


def qgemv_attn_prompt(dtype: int, head_dim: int, q_heads: int, kv_heads: int, q: int, q_token_stride: int,
                      q_head_stride: int, k: int, k_token_stride: int, k_head_stride: int, v: int,
                      v_token_stride: int, v_head_stride: int, n_seqs: int, cu_q: int, cu_k: int, n_q: int, n_k: int,
                      max_q: int, scale: float, out: int, out_token_stride: int, out_head_stride: int,
                      lse: int | None, ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_attn_prompt(dtype, head_dim, q_heads, kv_heads, q, q_token_stride, q_head_stride, k,
                                           k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, n_seqs,
                                           cu_q, cu_k, n_q, n_k, max_q, scale, out, out_token_stride, out_head_stride,
                                           lse, ws, ws_bytes, _stream_ptr(stream)))


# ----------------------------------------------------------- torch helper --

def _addr(a):
    """(address, keepalive) of a torch tensor / numpy array / None."""
    if a is None:
        return None, None
    if isinstance(a, np.ndarray):
        a = np.ascontiguousarray(a)
        return a.ctypes.data, a
    a = a.contiguous()
    return a.data_ptr(), a


def _current(stream):
    """The stream a torch-level call runs on: the one given, else torch's
    current stream (the C calls themselves take NULL as the legacy default
    stream)."""
    if stream is not None:
        return stream
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _along(stream, dev: int, make):
    """make() with `stream` as torch's current one, where one is given: what
    it allocates is memory of that stream, free of other streams' unfinished
    work, and the tensors that it returns (one, or a tuple) are not handed out
    again while the stream that was current still uses them."""
    torch = _torch()
    if stream is None:
        return make()
    ptr = _stream_ptr(stream)
    if ptr == torch._C._cuda_getCurrentRawStream(dev):
        return make()
    with torch.cuda.stream(torch.cuda.ExternalStream(ptr, device=dev) if ptr else torch.cuda.default_stream(dev)):
        out = make()
    before = torch.cuda.current_stream(dev)
    for t in out if isinstance(out, tuple) else (out,):
        t.record_stream(before)
    return out


def _empty_on(stream, dev: int):
    """torch.empty for a call on `stream`."""
    empty = _torch().empty
    return lambda *args, **kw: _along(stream, dev, lambda: empty(*args, **kw))


class QGemv:
    """One packed weight matrix on the GPU.

    ``QGemv(fmt, N, K, packed, scales=None, codebooks=None)`` copies the
    canonical inputs into the library; ``gemv(x)`` returns y = x . W^T as a
    new fp32 CUDA tensor, ``run(x, y)`` writes into ``y``.  Runs are ordered
    on ``stream`` when one is given, else on torch's current stream, like the
    torch operations around them."""

    def __init__(self, fmt, N: int, K: int, packed, scales=None, codebooks=None):
        self.fmt, self.N, self.K = _fmt(fmt), int(N), int(K)
        p, kp = _addr(packed)
        s, ks = _addr(scales)
        c, kc = _addr(codebooks)
        self.handle = qgemv_create(self.fmt, self.N, self.K, p, s, c)
        del kp, ks, kc

    @classmethod
    def stacked(cls, fmt, seg_rows, K: int, packed, scales=None, codebooks=None):
        """One handle over projections with the same K (rows stacked in
        order, codebook s for segment s; AQLM 2x8: a codebook pair per
        segment, the N row scales in order, segments on 2048-row blocks):
        one run computes them all."""
        self = cls.__new__(cls)
        self.fmt, self.N, self.K = _fmt(fmt), int(sum(seg_rows)), int(K)
        p, kp = _addr(packed)
        s, ks = _addr(scales)
        c, kc = _addr(codebooks)
        self.handle = qgemv_create_stacked(self.fmt, list(seg_rows), self.K, p, s, c)
        del kp, ks, kc
        return self

    @classmethod
    def glu(cls, fmt, N: int, K: int, packed_gate, packed_up, codebooks_gate=None, codebooks_up=None):
        """Fused MLP gate/up: ``gemv(x)`` returns SiLU(x . G^T) * (x . U^T),
        fp32 [M, N] (codebooks: each matrix's fp16 codebook for CBK4 / CBK8,
        CBK4_ROW's per-row fp32 [N, 16] arrays)."""
        self = cls.__new__(cls)
        self.fmt, self.N, self.K = _fmt(fmt), int(N), int(K)
        g, kg = _addr(packed_gate)
        u, ku = _addr(packed_up)
        cg, kcg = _addr(codebooks_gate)
        cu, kcu = _addr(codebooks_up)
        self.handle = qgemv_create_glu(self.fmt, self.N, self.K, g, u, cg, cu)
        del kg, ku, kcg, kcu
        return self

    def run(self, x, y, stream=None):
        M = x.shape[0]
        qgemv_run(self.handle, x.data_ptr(), M, y.data_ptr(), _current(stream))
        return y

    def run_residual(self, x, y, residual, stream=None):
        """y = residual + x . W^T (residual may be y itself)."""
        qgemv_run_residual(self.handle, x.data_ptr(), x.shape[0], y.data_ptr(), residual.data_ptr(),
                           _current(stream))
        return y

    def gemv(self, x, stream=None):
        import torch

        def make():
            y = torch.empty((x.shape[0], self.N), dtype=torch.float32, device=x.device)
            return self.run(x.contiguous(), y)
        return _along(stream, x.get_device(), make)

    def dequant(self, stream=None):
        import torch

        def make():
            w = torch.empty((self.N, self.K), dtype=torch.float32, device="cuda")
            qgemv_dequant(self.handle, w.data_ptr(), _current(None))
            return w
        return _along(stream, _device_now(), make)

    def status(self):
        return qgemv_status(self.handle)

    def set_batch_invariant(self, on: bool = True):
        qgemv_set_batch_invariant(self.handle, on)

    def set_x_int8(self, on: bool = True):
        qgemv_set_x_int8(self.handle, on)

    def run_xq(self, xq, M: int, y, residual=None, stream=None):
        """y (+ residual) from prepared INT8 activations (``prepare_x_int8``)."""
        qgemv_run_xq(self.handle, xq.data_ptr(), M, y.data_ptr(),
                     None if residual is None else residual.data_ptr(), _current(stream))
        return y

    def close(self):
        if getattr(self, "handle", None):
            qgemv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def quantize_q4_0(w, stream=None):
    """Q4_0 quantizer on the GPU: fp32 CUDA tensor [N, K] -> uint8 CUDA tensor."""
    import torch
    N, K = w.shape

    def make():
        out = torch.empty(qgemv_packed_bytes(Q4_0, N, K), dtype=torch.uint8, device=w.device)
        qgemv_quantize_q4_0(w.contiguous().data_ptr(), N, K, out.data_ptr(), _current(None))
        return out
    return _along(stream, w.get_device(), make)


def quantize_x_int8(x, stream=None):
    """PQ2_0 INT8 activation quantizer on the GPU: fp16 CUDA tensor [M, K]
    -> (int8 [M, K], fp32 scales [M, K/128]) CUDA tensors."""
    import torch
    M, K = x.shape

    def make():
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        a = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
        qgemv_quantize_x_int8(x.contiguous().data_ptr(), M, K, q.data_ptr(), a.data_ptr(), _current(None))
        return q, a
    return _along(stream, x.get_device(), make)


def prepare_x_int8(x, hadamard_block: int = 0, signs=None, stream=None):
    """PQ2_0 activation prologue on the GPU: fp16 CUDA tensor [M, K] -> the
    prepared uint8 CUDA buffer of ``qgemv_xq_bytes(M, K)`` bytes (INT8 codes in
    staging order, group scales, group code sums), after the Hadamard mixing
    of blocks of 1024 when ``hadamard_block`` is 1024 (signs: int8 CUDA
    tensor [K] of +-1, or None)."""
    import torch
    M, K = x.shape

    def make():
        xq = torch.empty(qgemv_xq_bytes(M, K), dtype=torch.uint8, device=x.device)
        qgemv_prepare_x_int8(x.contiguous().data_ptr(), M, K, None if signs is None else signs.data_ptr(),
                             hadamard_block, xq.data_ptr(), _current(None))
        return xq
    return _along(stream, x.get_device(), make)


# --------------------------------------------------- cache and attention --

# These calls run once a layer and token, so the host's time counts: what can be
# looked up once is (an import statement or an attribute chain each cost as much
# as a check).
_TORCH = None
_DTYPES = None  # torch dtype -> DT_*, filled on first use (torch is imported only where it is used)


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _on(stream, dev: int):
    """The address of the stream given, or of torch's current one of the device."""
    return _raw_stream(dev) if stream is None else _stream_ptr(stream)


def _raw_stream(dev: int) -> int:
    global _raw_stream  # torch's function itself, from the second call on
    _raw_stream = _torch()._C._cuda_getCurrentRawStream
    return _raw_stream(dev)


def _device_now() -> int:
    global _device_now
    _device_now = _torch()._C._cuda_getDevice
    return _device_now()


def _call(dev: int, fn, *args):
    """A library call with device `dev` current."""
    if dev == _device_now():
        rc = fn(*args)
    else:
        with _torch().cuda.device(dev):
            rc = fn(*args)
    return _check(rc) if rc else rc


def _gpu(what, device) -> None:
    if _torch().device(device).type != "cuda":
        raise ValueError(f"{what} must be on a CUDA device, not {device}")


def _dtype_code(dtype) -> int:
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: DT_F32, torch.float16: DT_F16, torch.bfloat16: DT_BF16}
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"rows are fp32, fp16 or bf16, not {dtype}")
    return code


def _where(dev) -> str:
    return "" if dev is None else f" on cuda:{dev}"


def _rows(name, t, heads: int, head_dim: int, dev: int | None = None):
    """(address, token stride, head stride) of a CUDA tensor [n, heads, head_dim], its values contiguous; on device `dev`
    where one is given."""
    shape, strides = t.shape, t.stride()
    if (len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or strides[2] != 1
            or (not t.is_cuda if dev is None else t.get_device() != dev)):
        raise ValueError(f"{name} must be a CUDA tensor [n, {heads}, {head_dim}] with contiguous values"
                         f"{_where(dev)}, got {tuple(shape)} with strides {strides} on {t.device}")
    # the stride of a dimension of one element means nothing to torch
    return (t.data_ptr(), strides[0] if shape[0] > 1 else heads * head_dim, strides[1] if heads > 1 else head_dim)


def _index(name, t, dtype, shape, dev: int | None = None):
    if (t.dtype != dtype or t.shape != shape or not t.is_contiguous()
            or (not t.is_cuda if dev is None else t.get_device() != dev)):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {shape}{_where(dev)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _elsewhere(workspace, dev: int):
    raise ValueError(f"the workspace must be on cuda:{dev}, not cuda:{workspace._dev}")


class AttnWorkspace:
    """Workspace of ``KVCache.attend`` and ``attn_prompt`` for up to
    ``n_seqs`` sequences, reused by any number of calls, one at a time (calls
    that overlap on several streams need one each).  Making one waits for its
    setting up on the current stream."""

    def __init__(self, n_seqs: int, q_heads: int, head_dim: int, device="cuda"):
        import torch
        self.nbytes = qgemv_attn_ws_bytes(n_seqs, q_heads, head_dim)
        if self.nbytes == 0:
            raise QgemvError(QGEMV_ERR_ARG, f"no workspace for {n_seqs} sequences of {q_heads} heads of {head_dim}")
        _gpu("a workspace", device)
        self.buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.ptr, self._dev = self.buffer.data_ptr(), self.buffer.get_device()
        self.reset()
        # The first call may be on another stream: what it counts on must be there.
        # (While a graph is captured the setting up is part of it.)
        stream = torch.cuda.current_stream(self._dev)
        with torch.cuda.stream(stream):
            if not torch.cuda.is_current_stream_capturing():
                stream.synchronize()

    def reset(self, stream=None):
        """Set the workspace up again (needed only after ``status`` raised)."""
        _call(self._dev, _lib.qgemv_attn_ws_init, self.ptr, self.nbytes, _on(stream, self._dev))

    def status(self):
        """Synchronise; raises if a kernel of this workspace gave up a wait."""
        return _call(self._dev, _lib.qgemv_attn_status, self.ptr)


class KVCache:
    """A paged key/value cache of one layer on the GPU.

    ``KVCache(fmt, n_pages, page_tokens, kv_heads, head_dim)`` with fmt "f16",
    "int8" or "q4_0" allocates (uninitialised) pages; ``write`` quantises new
    rows into slots, ``read`` gives rows back, ``attend`` is the attention of
    one or several drafted tokens of each sequence over the cached ones.
    Runs are ordered on ``stream`` when one is given, else on torch's current
    stream; outputs that a call makes are memory of that stream.  Tensors and
    workspace are on the cache's device, which need not be the current one."""

    def __init__(self, fmt, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int, device="cuda"):
        import torch
        self.fmt = _kv_fmt(fmt)
        self.kv_heads, self.head_dim, self.page_tokens, self.n_pages = kv_heads, head_dim, page_tokens, n_pages
        nbytes = qgemv_kv_bytes(self.fmt, n_pages, page_tokens, kv_heads, head_dim)
        if nbytes == 0:
            raise QgemvError(QGEMV_ERR_ARG, f"invalid cache: {fmt}, {n_pages} pages of {page_tokens} tokens, "
                                            f"{kv_heads} heads of {head_dim}")
        _gpu("a cache", device)
        self.pages = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.desc = KvCacheDesc(self.pages.data_ptr(), self.fmt, head_dim, kv_heads, page_tokens, n_pages)
        self._ref, self.device, self._dev = ctypes.byref(self.desc), self.pages.device, self.pages.get_device()

    def write(self, k, v, slots, stream=None):
        """Quantise the rows k and v [n, kv_heads, head_dim] (fp32, fp16 or
        bf16, any token and head strides) into slots (int64 [n]; a slot is
        page * page_tokens + place, negative ones are skipped)."""
        if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have the same type and number of tokens")
        n, dev = k.shape[0], self._dev
        s = _index("slots", slots, _torch().int64, (n,), dev)
        _call(dev, _lib.qgemv_kv_write, self._ref, _dtype_code(k.dtype), *_rows("k", k, self.kv_heads, self.head_dim, dev),
              *_rows("v", v, self.kv_heads, self.head_dim, dev), s, n, _on(stream, dev))

    def read(self, table, starts, cu, n_tokens: int, dtype=None, out=None, stream=None):
        """The cached rows of positions starts[b] .. of each sequence, packed
        by cu (int32 [n_seqs + 1]): (k, v) [n_tokens, kv_heads, head_dim] of
        dtype (fp16 unless given).  table: int32 [n_seqs, most pages]."""
        torch, dev = _torch(), self._dev
        n_seqs, stride = table.shape
        if out is None:
            shape = n_tokens, self.kv_heads, self.head_dim
            dtype = torch.float16 if dtype is None else dtype
            empty = torch.empty if stream is None else _empty_on(stream, dev)
            out = empty(shape, dtype=dtype, device=self.device), empty(shape, dtype=dtype, device=self.device)
            row = self.kv_heads * self.head_dim, self.head_dim
            rows = (out[0].data_ptr(), *row, out[1].data_ptr(), *row)
        else:
            k, v = out
            if k.dtype != v.dtype or k.shape[0] != n_tokens or v.shape[0] != n_tokens:
                raise ValueError(f"the outputs must have {n_tokens} tokens of one type")
            dtype = k.dtype
            rows = *_rows("k", k, self.kv_heads, self.head_dim, dev), *_rows("v", v, self.kv_heads, self.head_dim, dev)
        _call(dev, _lib.qgemv_kv_read, self._ref, _index("table", table, torch.int32, (n_seqs, stride), dev), stride, n_seqs,
              None if starts is None else _index("starts", starts, torch.int32, (n_seqs,), dev),
              _index("cu", cu, torch.int32, (n_seqs + 1,), dev), n_tokens, _dtype_code(dtype), *rows, _on(stream, dev))
        return out

    def attend(self, q, table, ctx_lens, cu_q, masks=None, *, max_ctx: int, max_new: int, workspace, scale=None,
               out=None, lse=None, stream=None):
        """Attention of the drafted tokens q [n, q_heads, head_dim] (fp16),
        which are in the cache at positions ctx_lens[b] + i of their
        sequences, over the first ctx_lens[b] positions and, by masks (int64
        or uint64 [n]: bit j for drafted token j; None: a chain), over one
        another.  Returns (out like q, lse fp32 [n, q_heads]).  scale is
        1 / sqrt(head_dim) unless given; max_ctx and max_new bound the
        lengths (they guide the split only)."""
        torch, dev = _torch(), self._dev
        n, heads, d = q.shape
        if q.dtype != torch.float16:
            raise ValueError("q must be fp16")
        if workspace._dev != dev:
            _elsewhere(workspace, dev)
        empty = torch.empty if stream is None else _empty_on(stream, dev)
        if out is None:
            out = empty((n, heads, d), dtype=torch.float16, device=self.device)
            out_rows = out.data_ptr(), heads * d, d
        elif out.dtype != torch.float16 or out.shape != q.shape:
            raise ValueError("out must be fp16, shaped like q")
        else:
            out_rows = _rows("out", out, heads, d, dev)
        if lse is None:
            lse = empty((n, heads), dtype=torch.float32, device=self.device)
        else:
            _index("lse", lse, torch.float32, (n, heads), dev)
        if masks is not None:
            masks = _index("masks", masks, torch.uint64 if masks.dtype == torch.uint64 else torch.int64, (n,), dev)
        n_seqs, stride = table.shape
        _call(dev, _lib.qgemv_attn_tree, self._ref, _index("table", table, torch.int32, (n_seqs, stride), dev), stride,
              n_seqs, _index("ctx_lens", ctx_lens, torch.int32, (n_seqs,), dev),
              *_rows("q", q, heads, self.head_dim, dev), heads, _index("cu_q", cu_q, torch.int32, (n_seqs + 1,), dev), n,
              masks, max_ctx, max_new, d ** -0.5 if scale is None else scale, *out_rows, lse.data_ptr(),
              workspace.ptr, workspace.nbytes, _on(stream, dev))
        return out, lse


def attn_prompt(q, k, v, cu_q, cu_k, *, max_q: int, workspace, scale=None, out=None, lse=None, stream=None):
    """Causal attention over packed prompts: q [n_q, q_heads, d], k and v
    [n_k, kv_heads, d] (all fp16 or all bf16), sequence b the rows cu_q[b] ..
    of q and cu_k[b] .. of k and v (int32 [n_seqs + 1]); its last query sees
    all of its keys.  max_q bounds the queries of a sequence: results are right
    whatever it is.  Returns (out like q, lse fp32 [n_q, q_heads]).  All
    tensors and the workspace are on q's device."""
    torch = _torch()
    n, heads, d = q.shape
    q_rows, dev = _rows("q", q, heads, d), q.get_device()
    if k.shape[0] != v.shape[0] or not (q.dtype == k.dtype == v.dtype):
        raise ValueError("q, k and v must have one type, k and v the same number of tokens")
    if workspace._dev != dev:
        _elsewhere(workspace, dev)
    empty = torch.empty if stream is None else _empty_on(stream, dev)
    if out is None:
        out = empty((n, heads, d), dtype=q.dtype, device=q.device)
        out_rows = out.data_ptr(), heads * d, d
    elif out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must have q's type and shape")
    else:
        out_rows = _rows("out", out, heads, d, dev)
    if lse is None:
        lse = empty((n, heads), dtype=torch.float32, device=q.device)
    else:
        _index("lse", lse, torch.float32, (n, heads), dev)
    n_seqs, kv_heads = cu_q.shape[0] - 1, k.shape[1]
    _call(dev, _lib.qgemv_attn_prompt, _dtype_code(q.dtype), d, heads, kv_heads, *q_rows,
          *_rows("k", k, kv_heads, d, dev), *_rows("v", v, kv_heads, d, dev), n_seqs,
          _index("cu_q", cu_q, torch.int32, (n_seqs + 1,), dev), _index("cu_k", cu_k, torch.int32, (n_seqs + 1,), dev), n,
          k.shape[0], max_q or 1, d ** -0.5 if scale is None else scale, *out_rows, lse.data_ptr(), workspace.ptr,
          workspace.nbytes, _on(stream, dev))
    return out, lse
