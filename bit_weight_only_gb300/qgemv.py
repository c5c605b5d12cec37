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
ROPE_HALVES, ROPE_NEIGHBOURS = 0, 1
ROPE_PAIRINGS = {"halves": ROPE_HALVES, "neighbours": ROPE_NEIGHBOURS}


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
    "qgemv_rope_plan_bytes": (_L, [_I]),
    "qgemv_rope_plan": (_I, [_P, _P, _I, _P]),
    "qgemv_rope_rows": (_I, [_P, _I, _I, _I, _P, _I, _I, _I, _P, _L, _L, _L, _I, _P, _L, _L, _P]),
    "qgemv_kv_write_rotated": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _L, _L, _I, _P, _L, _L, _P, _L, _L, _P, _L, _I,
                                    _P, _L, _L, _P]),
    "qgemv_beam_ws_bytes": (_L, [_L, _I, _L, _I]),
    "qgemv_beam_select": (_I, [_I, _P, _L, _L, _P, _L, _I, _I, _P, _P, _P, _P, _L, _P]),
    "qgemv_pool_reserve": (_I, [_P, _L, _I, _P, _L, _L, _P, _P, _P, _P]),
    "qgemv_pool_fork": (_I, [_P, _L, _I, _P, _L, _L, _P, _L, _P, _P, _P, _P, _P, _P, _P]),
    "qgemv_pool_release": (_I, [_P, _L, _I, _P, _L, _L, _P, _P, _P]),
    "qgemv_pool_ws_bytes": (_L, [_L]),
    "qgemv_pool_compact": (_I, [_P, _L, _P, _L, _L, _P, _P, _P, _L, _P, _L, _P]),
    "qgemv_kv_copy_pages": (_I, [_P, _P, _P, _P, _L, _P]),
    "qgemv_kv_summarize": (_I, [_P, _P, _L, _P, _P, _P]),
    "qgemv_kv_select_width": (_L, [_I, _L]),
    "qgemv_kv_select": (_I, [_P, _P, _P, _P, _L, _L, _P, _P, _L, _L, _I, _P, _L, _L, _P, _P, _P]),
    "qgemv_attn_pages": (_I, [_P, _P, _L, _L, _P, _P, _L, _L, _I, _P, _L, _P, _L, _L, _F, _P, _L, _L, _P, _P, _L, _P]),
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


def qgemv_rope_plan_bytes(pairs: int) -> int:
    return int(load().qgemv_rope_plan_bytes(pairs))


def qgemv_rope_plan(freqs: int, axes: int, pairs: int, plan: int) -> int:
    return _check(load().qgemv_rope_plan(freqs, axes, pairs, plan))


def qgemv_rope_rows(plan: int, pairs: int, pairing: int, n_axes: int, positions: int, dtype: int, heads: int,
                    head_dim: int, x: int, x_token_stride: int, x_head_stride: int, n_tokens: int, out_dtype: int,
                    out: int, out_token_stride: int, out_head_stride: int, stream=None) -> int:
    return _check(load().qgemv_rope_rows(plan, pairs, pairing, n_axes, positions, dtype, heads, head_dim, x,
                                         x_token_stride, x_head_stride, n_tokens, out_dtype, out, out_token_stride,
                                         out_head_stride, _stream_ptr(stream)))


def qgemv_kv_write_rotated(cache: KvCacheDesc, plan: int, pairs: int, pairing: int, n_axes: int, positions: int,
                           dtype: int, q: int, q_token_stride: int, q_head_stride: int, q_heads: int, k: int,
                           k_token_stride: int, k_head_stride: int, v: int, v_token_stride: int, v_head_stride: int,
                           slots: int, n_tokens: int, out_dtype: int, q_out: int, out_token_stride: int,
                           out_head_stride: int, stream=None) -> int:
    return _check(load().qgemv_kv_write_rotated(
        ctypes.byref(cache), plan, pairs, pairing, n_axes, positions, dtype, q, q_token_stride, q_head_stride, q_heads, k,
        k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, slots, n_tokens, out_dtype, q_out,
        out_token_stride, out_head_stride, _stream_ptr(stream)))


def qgemv_beam_ws_bytes(n_seqs: int, beams: int, vocab: int, width: int) -> int:
    return int(load().qgemv_beam_ws_bytes(n_seqs, beams, vocab, width))


def qgemv_beam_select(dtype: int, logits: int, row_stride: int, vocab: int, scores: int, n_seqs: int, beams: int, width: int,
                      out_scores: int, out_beams: int, out_tokens: int, ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_beam_select(dtype, logits, row_stride, vocab, scores, n_seqs, beams, width, out_scores,
                                           out_beams, out_tokens, ws, ws_bytes, _stream_ptr(stream)))


def qgemv_pool_reserve(refs: int, n_pages: int, page_tokens: int, table: int, table_stride: int, n_seqs: int, have: int,
                       need: int, state: int, stream=None) -> int:
    return _check(load().qgemv_pool_reserve(refs, n_pages, page_tokens, table, table_stride, n_seqs, have, need, state,
                                            _stream_ptr(stream)))


def qgemv_pool_fork(refs: int, n_pages: int, page_tokens: int, table: int, table_stride: int, n_rows: int, parents: int,
                    n_new: int, lens: int, new_table: int, src: int, dst: int, tokens: int, state: int, stream=None) -> int:
    return _check(load().qgemv_pool_fork(refs, n_pages, page_tokens, table, table_stride, n_rows, parents, n_new, lens,
                                         new_table, src, dst, tokens, state, _stream_ptr(stream)))


def qgemv_pool_release(refs: int, n_pages: int, page_tokens: int, table: int, table_stride: int, n_seqs: int, lens: int,
                       keep: int | None, stream=None) -> int:
    return _check(load().qgemv_pool_release(refs, n_pages, page_tokens, table, table_stride, n_seqs, lens, keep,
                                            _stream_ptr(stream)))


def qgemv_pool_ws_bytes(n_pages: int) -> int:
    return int(load().qgemv_pool_ws_bytes(n_pages))


def qgemv_pool_compact(refs: int, n_pages: int, table: int, table_stride: int, n_seqs: int, new_table: int, src: int, dst: int,
                       n_moves: int, ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_pool_compact(refs, n_pages, table, table_stride, n_seqs, new_table, src, dst, n_moves, ws,
                                            ws_bytes, _stream_ptr(stream)))


def qgemv_kv_copy_pages(cache: KvCacheDesc, src: int, dst: int, tokens: int | None, n: int, stream=None) -> int:
    return _check(load().qgemv_kv_copy_pages(ctypes.byref(cache), src, dst, tokens, n, _stream_ptr(stream)))


def qgemv_kv_summarize(cache: KvCacheDesc, pages: int, n: int, codes: int, scales: int, stream=None) -> int:
    return _check(load().qgemv_kv_summarize(ctypes.byref(cache), pages, n, codes, scales, _stream_ptr(stream)))


def qgemv_kv_select_width(page_tokens: int, n_select: int) -> int:
    return int(load().qgemv_kv_select_width(page_tokens, n_select))


def qgemv_kv_select(cache: KvCacheDesc, codes: int, scales: int, table: int, table_stride: int, n_seqs: int, ctx_lens: int,
                    q: int, q_token_stride: int, q_head_stride: int, q_heads: int, cu_q: int, n_q: int, n_select: int,
                    pages: int, lens: int, stream=None) -> int:
    return _check(load().qgemv_kv_select(ctypes.byref(cache), codes, scales, table, table_stride, n_seqs, ctx_lens, q,
                                         q_token_stride, q_head_stride, q_heads, cu_q, n_q, n_select, pages, lens,
                                         _stream_ptr(stream)))


def qgemv_attn_pages(cache: KvCacheDesc, pages: int, pages_stride: int, n_seqs: int, ctx_lens: int, q: int,
                     q_token_stride: int, q_head_stride: int, q_heads: int, cu_q: int, n_q: int, masks: int | None,
                     max_ctx: int, max_new: int, scale: float, out: int, out_token_stride: int, out_head_stride: int,
                     lse: int | None, ws: int, ws_bytes: int, stream=None) -> int:
    return _check(load().qgemv_attn_pages(ctypes.byref(cache), pages, pages_stride, n_seqs, ctx_lens, q, q_token_stride,
                                          q_head_stride, q_heads, cu_q, n_q, masks, max_ctx, max_new, scale, out,
                                          out_token_stride, out_head_stride, lse, ws, ws_bytes, _stream_ptr(stream)))


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


def _settle(dev: int) -> None:
    """Wait for what the current stream sets up, so that any stream may use it first (while a graph is captured the
    setting up is part of it)."""
    torch = _torch()
    stream = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        if not torch.cuda.is_current_stream_capturing():
            stream.synchronize()


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
    if (len(shape) != 3 or shape[1] != heads or shape[2] != head_dim or (strides[2] != 1 and shape[0] > 0)
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


class Rotary:
    """Rotary positions for heads of head_dim values, on the GPU.

    ``Rotary(head_dim, sections, base=10000.0)``: sections[a] pairs of each
    head belong to axis a of a position (one to four axes; ``[head_dim // 2]``
    for plain text); with n pairs in all, pair j turns by
    ``position[axis(j)] * base ** (-j / n)``, or by ``freqs[j]`` a position
    where those are given.  pairs: "halves" (values j and j + n are a pair) or
    "neighbours" (2j and 2j + 1).  Values behind the pairs stay.  ``rotate``
    turns rows, ``KVCache.write_rotated`` turns q and k on their way into a
    cache; negative positions turn back."""

    def __init__(self, head_dim: int, sections, base: float = 10000.0, freqs=None, pairs: str = "halves", device="cuda"):
        import torch
        sections = [int(s) for s in sections]
        n = sum(sections)
        if head_dim not in (64, 128) or not 1 <= len(sections) <= 4 or min(sections) < 0 or not 1 <= n <= head_dim // 2:
            raise QgemvError(QGEMV_ERR_ARG, f"invalid plan: sections {sections} of a head of {head_dim}")
        if pairs not in ROPE_PAIRINGS:
            raise QgemvError(QGEMV_ERR_ARG, f"unknown pairing {pairs!r}")
        freqs = [float(base) ** (-j / n) for j in range(n)] if freqs is None else [float(f) for f in freqs]
        if len(freqs) != n:
            raise QgemvError(QGEMV_ERR_ARG, f"{len(freqs)} frequencies for {n} pairs")
        f = np.array(freqs, dtype=np.float64)
        a = np.repeat(np.arange(len(sections), dtype=np.int32), sections)
        plan = np.zeros(qgemv_rope_plan_bytes(n) // 8, dtype=np.int64)
        qgemv_rope_plan(f.ctypes.data, a.ctypes.data, n, plan.ctypes.data)
        _gpu("a rotary plan", device)
        self.head_dim, self.pairs, self.axes, self.pairing = head_dim, n, len(sections), ROPE_PAIRINGS[pairs]
        self.plan = torch.from_numpy(plan).to(device)
        self.ptr, self._dev = self.plan.data_ptr(), self.plan.get_device()
        _settle(self._dev)

    def rotate(self, x, positions, dtype=None, out=None, stream=None):
        """The rows x [n, heads, head_dim] turned to the positions (int32 [n,
        axes]), of x's type unless dtype is given; out may be x itself, but no
        other rows that overlap x."""
        n, heads, d = x.shape
        dev = self._dev
        rows = _rows("x", x, heads, self.head_dim, dev)
        if out is None:
            torch = _torch()
            empty = torch.empty if stream is None else _empty_on(stream, dev)
            out = empty((n, heads, d), dtype=x.dtype if dtype is None else dtype, device=x.device)
            out_rows = out.data_ptr(), heads * d, d
        elif out.shape != x.shape or dtype not in (None, out.dtype):
            raise ValueError("out must be shaped like x, of the dtype given")
        else:
            out_rows = _rows("out", out, heads, d, dev)
        _call(dev, _lib.qgemv_rope_rows, self.ptr, self.pairs, self.pairing, self.axes,
              _index("positions", positions, _torch().int32, (n, self.axes), dev), _dtype_code(x.dtype), heads, d, *rows, n,
              _dtype_code(out.dtype), *out_rows, _on(stream, dev))
        return out


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

    def write_rotated(self, rotary, q, k, v, positions, slots, out=None, stream=None):
        """``write`` of k rotated to the positions (int32 [n, axes]) and v as
        it is, and q [n, q_heads, head_dim] rotated, in one launch; q, k and v
        have one type.  Returns the rotated q: fp16, or of the type of ``out``."""
        torch, dev = _torch(), self._dev
        n, heads, d = q.shape
        if not q.dtype == k.dtype == v.dtype or k.shape[0] != n or v.shape[0] != n:
            raise ValueError("q, k and v must have the same type and number of tokens")
        if rotary._dev != dev or rotary.head_dim != self.head_dim:
            raise ValueError(f"the rotary plan is for heads of {rotary.head_dim} on cuda:{rotary._dev}, the cache has "
                             f"heads of {self.head_dim} on cuda:{dev}")
        if out is None:
            empty = torch.empty if stream is None else _empty_on(stream, dev)
            out = empty((n, heads, d), dtype=torch.float16, device=self.device)
            out_rows = out.data_ptr(), heads * d, d
        elif out.shape != q.shape:
            raise ValueError("out must be shaped like q")
        else:
            out_rows = _rows("out", out, heads, d, dev)
        _call(dev, _lib.qgemv_kv_write_rotated, self._ref, rotary.ptr, rotary.pairs, rotary.pairing, rotary.axes,
              _index("positions", positions, torch.int32, (n, rotary.axes), dev), _dtype_code(q.dtype),
              *_rows("q", q, heads, self.head_dim, dev), heads, *_rows("k", k, self.kv_heads, self.head_dim, dev),
              *_rows("v", v, self.kv_heads, self.head_dim, dev), _index("slots", slots, torch.int64, (n,), dev), n,
              _dtype_code(out.dtype), *out_rows, _on(stream, dev))
        return out

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

    def copy_pages(self, src, dst, tokens=None, stream=None):
        """Copy page src[i] to page dst[i] (int32 [n]), whole or the first
        tokens[i] tokens (int32 [n]); pairs with a number that is no page are
        passed over.  No page may be the destination of two copies, or of one
        and the source of another."""
        dev, i32 = self._dev, _torch().int32
        n, = src.shape
        _call(dev, _lib.qgemv_kv_copy_pages, self._ref, _index("src", src, i32, (n,), dev), _index("dst", dst, i32, (n,), dev),
              None if tokens is None else _index("tokens", tokens, i32, (n,), dev), n, _on(stream, dev))

    def attend(self, q, table, ctx_lens, cu_q, masks=None, *, max_ctx: int, max_new: int, workspace, scale=None,
               out=None, lse=None, stream=None):
        """Attention of the drafted tokens q [n, q_heads, head_dim] (fp16),
        which are in the cache at positions ctx_lens[b] + i of their
        sequences, over the first ctx_lens[b] positions and, by masks (int64
        or uint64 [n]: bit j for drafted token j; None: a chain), over one
        another.  Returns (out like q, lse fp32 [n, q_heads]).  scale is
        1 / sqrt(head_dim) unless given; max_ctx and max_new bound the
        lengths (they guide the split only)."""
        n_seqs, stride = table.shape
        return self._attend(_lib.qgemv_attn_tree, _index("table", table, _torch().int32, (n_seqs, stride), self._dev), n_seqs,
                            stride, q, ctx_lens, cu_q, masks, max_ctx, max_new, workspace, scale, out, lse, stream)

    def select(self, q, table, ctx_lens, cu_q, *, summary, n_select: int, out=None, stream=None):
        """For each sequence and key/value head the n_select whole pages of
        highest score (``KeySummary``) before ctx_lens[b], in order, and the
        pages behind them: (pages int32 [n_seqs, kv_heads, width], lens int32
        [n_seqs]), a page table of each head's own and the context's length
        over it, for ``attend_pages``.  q, table, ctx_lens and cu_q as for
        ``attend``."""
        torch, dev = _torch(), self._dev
        n, heads, d = q.shape
        if q.dtype != torch.float16:
            raise ValueError("q must be fp16")
        if summary.cache is not self:
            raise ValueError("the summary is another cache's")
        n_seqs, stride = table.shape
        width = _lib.qgemv_kv_select_width(self.page_tokens, n_select)
        if width == 0:
            raise QgemvError(QGEMV_ERR_ARG, f"n_select={n_select} is not in [0, 2^20]")
        if out is None:
            empty = torch.empty if stream is None else _empty_on(stream, dev)
            pages = empty((n_seqs, self.kv_heads, width), dtype=torch.int32, device=self.device)
            lens = empty((n_seqs,), dtype=torch.int32, device=self.device)
            out, to = (pages, lens), (pages.data_ptr(), lens.data_ptr())
        else:
            to = (_index("pages", out[0], torch.int32, (n_seqs, self.kv_heads, width), dev),
                  _index("lens", out[1], torch.int32, (n_seqs,), dev))
        _call(dev, _lib.qgemv_kv_select, self._ref, summary.codes.data_ptr(), summary.scales.data_ptr(),
              _index("table", table, torch.int32, (n_seqs, stride), dev), stride, n_seqs,
              _index("ctx_lens", ctx_lens, torch.int32, (n_seqs,), dev), *_rows("q", q, heads, self.head_dim, dev), heads,
              _index("cu_q", cu_q, torch.int32, (n_seqs + 1,), dev), n, n_select, *to, _on(stream, dev))
        return out

    def attend_pages(self, q, pages, lens, cu_q, masks=None, *, max_ctx: int, max_new: int, workspace, scale=None, out=None,
                     lse=None, stream=None):
        """``attend`` with a page table for each key/value head: pages int32
        [n_seqs, kv_heads, width] and the contexts' lengths over it, as
        ``select`` gives them."""
        n_seqs, heads, stride = pages.shape
        return self._attend(_lib.qgemv_attn_pages, _index("pages", pages, _torch().int32, (n_seqs, self.kv_heads, stride), self._dev),
                            n_seqs, stride, q, lens, cu_q, masks, max_ctx, max_new, workspace, scale, out, lse, stream)

    def _attend(self, fn, table, n_seqs, stride, q, ctx_lens, cu_q, masks, max_ctx, max_new, workspace, scale, out, lse, stream):
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
        _call(dev, fn, self._ref, table, stride, n_seqs, _index("ctx_lens", ctx_lens, torch.int32, (n_seqs,), dev),
              *_rows("q", q, heads, self.head_dim, dev), heads, _index("cu_q", cu_q, torch.int32, (n_seqs + 1,), dev), n,
              masks, max_ctx, max_new, d ** -0.5 if scale is None else scale, *out_rows, lse.data_ptr(),
              workspace.ptr, workspace.nbytes, _on(stream, dev))
        return out, lse


class KeySummary:
    """Summaries of a cache's pages, by which ``KVCache.select`` scores them:
    per page and key/value head the largest and smallest key values of each
    channel, as INT8 ``codes`` [n_pages, kv_heads, 2, head_dim] with a scale
    (``scales`` [n_pages, kv_heads]).  ``update`` takes those of pages that have
    become full; it has to be called again for pages that are written anew or
    copied to."""

    def __init__(self, cache: KVCache):
        import torch
        self.cache = cache
        shape = cache.n_pages, cache.kv_heads
        self.codes = torch.zeros(*shape, 2, cache.head_dim, dtype=torch.int8, device=cache.device)
        self.scales = torch.zeros(shape, dtype=torch.float32, device=cache.device)
        _settle(cache._dev)

    def update(self, pages, stream=None):
        """Take the summaries of the pages (int32 [n]; numbers that are no page
        of the cache are passed over)."""
        c = self.cache
        n, = pages.shape
        _call(c._dev, _lib.qgemv_kv_summarize, c._ref, _index("pages", pages, _torch().int32, (n,), c._dev), n,
              self.codes.data_ptr(), self.scales.data_ptr(), _on(stream, c._dev))


class PagePool:
    """The pages of one or more caches of n_pages pages (say a cache a layer,
    with one page table): ``refs`` (int32 [n_pages]) counts the rows of page
    tables that hold a page, 0 for a free one.  A row of n tokens holds the
    pages of its first ceil(n / page_tokens) entries.  ``reserve`` gives pages
    out, lowest first; ``fork`` makes the new rows of a step of beam search;
    ``release`` takes pages back; ``compact`` packs the pages in use.  Tables
    are int32 [rows, entries], lengths int32 [rows].  Calls return at once, and
    run one at a time; ``status`` tells whether pages ran out."""

    def __init__(self, n_pages: int, page_tokens: int, device="cuda"):
        import torch
        nbytes = qgemv_pool_ws_bytes(n_pages)
        if nbytes == 0 or page_tokens not in (16, 32, 64, 128, 256):
            raise QgemvError(QGEMV_ERR_ARG, f"invalid pool: {n_pages} pages of {page_tokens} tokens")
        _gpu("a pool", device)
        self.n_pages, self.page_tokens, self._nbytes = n_pages, page_tokens, nbytes
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=device)
        self._state = torch.zeros(2, dtype=torch.int32, device=device)  # pages that were missing; the calls' own
        self._ws = torch.empty(nbytes // 4, dtype=torch.int32, device=device)
        self._dev, self.device = self.refs.get_device(), self.refs.device
        _settle(self._dev)

    def _ints(self, name, t, *shape):
        return _index(name, t, _torch().int32, shape, self._dev)

    def reserve(self, table, have, need, stream=None):
        """Give row b, which holds have[b] tokens, the pages for need[b]; the
        table's entries are filled in place.  (Tokens past the table's width
        get none, and ``status`` does not tell.)"""
        rows, stride = table.shape
        _call(self._dev, _lib.qgemv_pool_reserve, self.refs.data_ptr(), self.n_pages, self.page_tokens,
              self._ints("table", table, rows, stride), stride, rows, self._ints("have", have, rows),
              self._ints("need", need, rows), self._state.data_ptr(), _on(stream, self._dev))

    def fork(self, table, parents, lens, stream=None):
        """Replace the rows of table (lens tokens each) by new ones, row r what
        row parents[r] (int32 [n]) was: whole pages are shared, rows without
        children return theirs.  Returns (new table, src, dst, tokens): the page
        that a row has filled in part stays with its first child, the others
        get one each, and ``copy_pages(src, dst, tokens)`` of every cache
        copies its tokens."""
        torch, dev = _torch(), self._dev
        i32 = torch.int32
        rows, stride = table.shape
        n, = parents.shape
        old = _index("table", table, i32, (rows, stride), dev)
        ups, ls = _index("parents", parents, i32, (n,), dev), _index("lens", lens, i32, (rows,), dev)
        if stream is None:
            like = torch.empty_like
            new = like(table) if n == rows else torch.empty((n, stride), dtype=i32, device=self.device)
            src, dst, tokens = like(parents), like(parents), like(parents)
        else:
            empty = _empty_on(stream, dev)
            new = empty((n, stride), dtype=i32, device=self.device)
            src, dst, tokens = (empty((n,), dtype=i32, device=self.device) for _ in range(3))
        _call(dev, _lib.qgemv_pool_fork, self.refs.data_ptr(), self.n_pages, self.page_tokens, old, stride, rows, ups, n, ls,
              new.data_ptr(), src.data_ptr(), dst.data_ptr(), tokens.data_ptr(), self._state.data_ptr(), _on(stream, dev))
        return new, src, dst, tokens

    def release(self, table, lens, keep=None, stream=None):
        """Take back the pages of row b's tokens keep[b] .. lens[b] (all of
        them unless keep is given) that no kept token is in; their entries
        become -1.  A page that is kept in part is still shared with the rows
        that hold it, and no call makes it the row's alone: a row that goes on
        from there writes into theirs."""
        rows, stride = table.shape
        _call(self._dev, _lib.qgemv_pool_release, self.refs.data_ptr(), self.n_pages, self.page_tokens,
              self._ints("table", table, rows, stride), stride, rows, self._ints("lens", lens, rows),
              None if keep is None else self._ints("keep", keep, rows), _on(stream, self._dev))

    def compact(self, table, out=None, stream=None):
        """Move the pages in use to the lowest numbers.  Returns (new table,
        src, dst): the moves, for ``copy_pages`` of every cache, end with -1.
        The table holds every row that is in use; out may be table itself."""
        torch, dev = _torch(), self._dev
        rows, stride = table.shape
        empty = torch.empty if stream is None else _empty_on(stream, dev)
        n = self.n_pages // 2
        if out is None:
            out = empty((rows, stride), dtype=torch.int32, device=self.device)
        src, dst = empty((n,), dtype=torch.int32, device=self.device), empty((n,), dtype=torch.int32, device=self.device)
        _call(dev, _lib.qgemv_pool_compact, self.refs.data_ptr(), self.n_pages, self._ints("table", table, rows, stride), stride,
              rows, self._ints("out", out, rows, stride), src.data_ptr(), dst.data_ptr(), n, self._ws.data_ptr(), self._nbytes,
              _on(stream, dev))
        return out, src, dst

    def status(self):
        """Synchronise; raises if pages ran out since the last call."""
        torch = _torch()
        torch.cuda.synchronize(self._dev)
        n = int(self._state[0].item())
        if n:
            self._state[0] = 0
            torch.cuda.synchronize(self._dev)
            raise QgemvError(QGEMV_ERR_NOMEM, f"{n} pages were not there to give")


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


class BeamWorkspace:
    """Workspace of ``beam_select`` for up to n_seqs sequences of these sizes,
    reused by any number of calls, one at a time (calls that overlap on several
    streams need one each)."""

    def __init__(self, n_seqs: int, beams: int, vocab: int, width: int, device="cuda"):
        import torch
        self.nbytes = qgemv_beam_ws_bytes(n_seqs, beams, vocab, width)
        if self.nbytes == 0:
            raise QgemvError(QGEMV_ERR_ARG, f"no workspace for {n_seqs} sequences of {beams} beams, {vocab} tokens, {width} kept")
        _gpu("a workspace", device)
        self.buffer = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        self.ptr, self._dev = self.buffer.data_ptr(), self.buffer.get_device()
        _settle(self._dev)


def beam_select(logits, scores, width: int, *, workspace, out=None, stream=None):
    """Beam search's choice: of each sequence's candidates (beam, token) the
    width with the largest scores[s, b] + log_softmax(logits)[token], in
    descending order, ties to the lower beam and token.  logits [n_seqs *
    beams, vocab] (fp32, fp16 or bf16, any row stride), scores fp32 [n_seqs,
    beams].  Returns (scores fp32, beams int32, tokens int32), each [n_seqs,
    width]; (-inf, -1, -1) where there is no candidate.  All tensors and the
    workspace are on the logits' device."""
    torch, dev = _torch(), logits.get_device()
    n_seqs, beams = scores.shape
    shape, strides = logits.shape, logits.stride()
    if len(shape) != 2 or shape[0] != n_seqs * beams or (strides[1] != 1 and shape[1] > 1) or not logits.is_cuda:
        raise ValueError(f"logits must be a CUDA tensor [{n_seqs * beams}, vocab] with contiguous rows, got {tuple(shape)} with "
                         f"strides {strides} on {logits.device}")
    if workspace._dev != dev:
        _elsewhere(workspace, dev)
    if out is None:
        empty = torch.empty if stream is None else _empty_on(stream, dev)
        best = empty((n_seqs, width), dtype=torch.float32, device=logits.device)
        parents = empty((n_seqs, width), dtype=torch.int32, device=logits.device)
        tokens = empty((n_seqs, width), dtype=torch.int32, device=logits.device)
        out, to = (best, parents, tokens), (best.data_ptr(), parents.data_ptr(), tokens.data_ptr())
    else:
        to = tuple(_index(f"out[{i}]", t, kind, (n_seqs, width), dev)
                   for i, (t, kind) in enumerate(zip(out, (torch.float32, torch.int32, torch.int32))))
    _call(dev, _lib.qgemv_beam_select, _dtype_code(logits.dtype), logits.data_ptr(), strides[0] if shape[0] > 1 else shape[1],
          shape[1], _index("scores", scores, torch.float32, (n_seqs, beams), dev), n_seqs, beams, width, *to, workspace.ptr,
          workspace.nbytes, _on(stream, dev))
    return out
