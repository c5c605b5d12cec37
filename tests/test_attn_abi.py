"""Host-side checks of the cache and attention calls (no GPU needed): sizes, and refusals before anything is launched."""
import ctypes

import pytest

from bit_weight_only_gb300 import build, qgemv

ARG, ALIGN, OK = qgemv.QGEMV_ERR_ARG, qgemv.QGEMV_ERR_ALIGN, qgemv.QGEMV_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qgemv.load()


def test_cache_sizes(lib):
    assert qgemv.qgemv_kv_bytes("f16", 3, 64, 8, 128) == 3 * 64 * 8 * 2 * 256
    assert qgemv.qgemv_kv_bytes("int8", 3, 16, 8, 128) == 3 * 16 * 8 * 2 * 132
    assert qgemv.qgemv_kv_bytes("q4_0", 3, 256, 1, 64) == 3 * 256 * 2 * 36
    assert qgemv.qgemv_kv_bytes("f16", 1 << 30, 256, 64, 128) == (1 << 30) * 256 * 64 * 512  # past 32 bits
    for bad in (("f16", 0, 64, 8, 128), ("f16", 1, 48, 8, 128), ("f16", 1, 512, 8, 128), ("f16", 1, 8, 8, 128),
                ("f16", 1, 64, 0, 128), ("f16", 1, 64, 8, 96), (0, 1, 64, 8, 128), (4, 1, 64, 8, 128)):
        assert qgemv.qgemv_kv_bytes(*bad) == 0


def test_workspace_sizes(lib):
    assert qgemv.qgemv_attn_ws_bytes(1, 32, 128) >= 256
    assert qgemv.qgemv_attn_ws_bytes(64, 32, 128) >= qgemv.qgemv_attn_ws_bytes(1, 32, 128)
    for bad in ((-1, 32, 128), (1, 0, 128), (1, 32, 80)):
        assert qgemv.qgemv_attn_ws_bytes(*bad) == 0
    assert lib.qgemv_attn_ws_init(None, 1 << 20, None) == ARG
    assert lib.qgemv_attn_ws_init(256, 8, None) == ARG
    assert lib.qgemv_attn_status(None) == ARG


def cache(**kw):
    d = {"pages": 4096, "format": qgemv.KV_INT8, "head_dim": 128, "kv_heads": 2, "page_tokens": 64, "n_pages": 4, **kw}
    return ctypes.byref(qgemv.KvCacheDesc(*[d[n] for n, _ in qgemv.KvCacheDesc._fields_]))


def call(fn, defaults, kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


WRITE = {"cache": None, "dtype": 1, "k": 256, "kt": 256, "kh": 128, "v": 256, "vt": 256, "vh": 128, "slots": 64, "n": 5,
         "stream": None}
READ = {"cache": None, "table": 64, "table_stride": 4, "n_seqs": 2, "starts": None, "cu": 64, "n": 5, "dtype": 1, "k": 256,
        "kt": 256, "kh": 128, "v": 256, "vt": 256, "vh": 128, "stream": None}
TREE = {"cache": None, "table": 64, "table_stride": 4, "n_seqs": 2, "ctx": 64, "q": 256, "qt": 1024, "qh": 128, "heads": 8,
        "cu": 64, "n": 5, "masks": None, "max_ctx": 100, "max_new": 3, "scale": 1.0, "out": 256, "ot": 1024, "oh": 128,
        "lse": None, "ws": 256, "ws_bytes": 1 << 40, "stream": None}
PROMPT = {"dtype": 1, "d": 128, "heads": 8, "kv_heads": 2, "q": 256, "qt": 1024, "qh": 128, "k": 256, "kt": 256, "kh": 128,
          "v": 256, "vt": 256, "vh": 128, "n_seqs": 2, "cu_q": 64, "cu_k": 64, "n_q": 5, "n_k": 5, "max_q": 5, "scale": 1.0,
          "out": 256, "ot": 1024, "oh": 128, "lse": None, "ws": 256, "ws_bytes": 1 << 40, "stream": None}

BAD_CACHE = [({"pages": None}, ARG), ({"pages": 4100}, ALIGN), ({"format": 9}, ARG), ({"head_dim": 96}, ARG),
             ({"page_tokens": 24}, ARG), ({"n_pages": 0}, ARG), ({"kv_heads": 0}, ARG)]


@pytest.mark.parametrize("bad, code", BAD_CACHE)
def test_bad_caches_are_refused(lib, bad, code):
    for fn, d in ((lib.qgemv_kv_write, WRITE), (lib.qgemv_kv_read, READ), (lib.qgemv_attn_tree, TREE)):
        assert call(fn, d, {"cache": cache(**bad)}) == code
        assert call(fn, d, {"cache": None}) == ARG


@pytest.mark.parametrize("kw, code", [({"dtype": 3}, ARG), ({"dtype": -1}, ARG), ({"k": None}, ARG), ({"v": None}, ARG),
                                      ({"slots": None}, ARG), ({"n": -1}, ARG), ({"k": 264}, ALIGN), ({"vt": 257}, ALIGN),
                                      ({"kh": 4}, ALIGN), ({"kt": -256}, ARG), ({"slots": 68}, ALIGN), ({"n": 0}, OK)])
def test_write_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_write, WRITE, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"dtype": 7}, ARG), ({"table": None}, ARG), ({"cu": None}, ARG), ({"k": None}, ARG),
                                      ({"n_seqs": -1}, ARG), ({"kt": 64}, ARG), ({"vh": 64}, ARG), ({"v": 258}, ALIGN),
                                      ({"cu": 66}, ALIGN), ({"n": 0}, OK), ({"n_seqs": 0}, OK)])
def test_read_refusals(lib, kw, code):
    assert call(lib.qgemv_kv_read, READ, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"heads": 7}, ARG), ({"heads": 0}, ARG), ({"q": None}, ARG), ({"out": None}, ARG),
                                      ({"ctx": None}, ARG), ({"cu": None}, ARG), ({"table": None}, ARG), ({"n": -3}, ARG),
                                      ({"max_ctx": -1}, ARG), ({"q": 260}, ALIGN), ({"ot": 100}, ARG), ({"oh": 120}, ARG),
                                      ({"qt": 1025}, ALIGN), ({"masks": 4}, ALIGN), ({"ws": None}, ARG), ({"ws": 264}, ALIGN),
                                      ({"ws_bytes": 100}, ARG), ({"lse": 2}, ALIGN), ({"n": 0}, OK), ({"n_seqs": 0}, OK)])
def test_tree_refusals(lib, kw, code):
    assert call(lib.qgemv_attn_tree, TREE, {"cache": cache(), **kw}) == code


@pytest.mark.parametrize("kw, code", [({"dtype": 0}, ARG), ({"d": 80}, ARG), ({"heads": 9}, ARG), ({"kv_heads": 0}, ARG),
                                      ({"q": None}, ARG), ({"k": None}, ARG), ({"out": None}, ARG), ({"cu_q": None}, ARG),
                                      ({"cu_k": None}, ARG), ({"n_q": -1}, ARG), ({"max_q": -1}, ARG), ({"k": 257}, ALIGN),
                                      ({"vt": 130}, ALIGN), ({"ot": 64}, ARG), ({"ws": None}, ARG), ({"ws_bytes": 1}, ARG),
                                      ({"cu_k": 65}, ALIGN), ({"kt": 0}, ARG), ({"vh": 0}, ARG), ({"qt": 0}, ARG),
                                      ({"heads": 258, "ot": 258 * 128}, ARG), ({"n_q": 0}, OK), ({"n_seqs": 0}, OK), ({"max_q": 0}, OK)])
def test_prompt_refusals(lib, kw, code):
    assert call(lib.qgemv_attn_prompt, PROMPT, kw) == code


def test_torch_level_refusals(lib):
    torch = pytest.importorskip("torch")
    t = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qgemv._rows("k", t, 2, 64)
    with pytest.raises(ValueError, match="fp32, fp16 or bf16"):
        qgemv._dtype_code(torch.int8)
    with pytest.raises(ValueError, match="cu"):
        qgemv._index("cu", torch.zeros(3), torch.int32, (3,))
    with pytest.raises(qgemv.QgemvError):
        qgemv.KVCache("int8", 1, 48, 2, 64, device="cpu")
    with pytest.raises(qgemv.QgemvError):
        qgemv.AttnWorkspace(1, 8, 80, device="cpu")
