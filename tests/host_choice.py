"""Runs library calls in a child process on a stand-in for the CUDA runtime (fake_cuda_runtime.c): what the host would launch,
on a machine without a GPU."""
import json
import os
import subprocess
import sys

from bit_weight_only_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))

PRELUDE = """
import ctypes, json, sys
sys.path.insert(0, {root!r})
from bit_weight_only_gb300 import qgemv
fake = ctypes.CDLL(None)
fake.fake_note.restype = ctypes.c_char_p
lib = qgemv.load()

def notes():
    got = [fake.fake_note(i).decode().split(" ") for i in range(fake.fake_notes())]
    fake.fake_clear()
    return got

def cache(fmt="int8", kv_heads=2, head_dim=128, page=64, n_pages=1 << 16):
    return ctypes.byref(qgemv.KvCacheDesc(4096, qgemv.KV_FORMATS[fmt], head_dim, kv_heads, page, n_pages))

def tree(fmt="int8", kv_heads=2, q_heads=8, head_dim=128, n_seqs=2, n=5, max_ctx=100, max_new=3, ot=None, oh=None):
    ot = q_heads * head_dim if ot is None else ot
    oh = head_dim if oh is None else oh
    return lib.qgemv_attn_tree(cache(fmt, kv_heads, head_dim), 64, 4, n_seqs, 64, 256, q_heads * head_dim, head_dim, q_heads,
                               64, n, None, max_ctx, max_new, 1.0, 256, ot, oh, None, 256, 1 << 40, None)

def prompt(dtype=1, head_dim=128, q_heads=8, kv_heads=2, n_seqs=1, n_q=4096, n_k=4096, ot=None, oh=None):
    q, k = q_heads * head_dim, kv_heads * head_dim
    return lib.qgemv_attn_prompt(dtype, head_dim, q_heads, kv_heads, 256, q, head_dim, 256, k, head_dim, 256, k, head_dim,
                                 n_seqs, 64, 64, n_q, n_k, n_q, 1.0, 256, q if ot is None else ot,
                                 head_dim if oh is None else oh, None, 256, 1 << 40, None)

def read(kv_heads=2, head_dim=128, n=5, kt=None, kh=None):
    kt = kv_heads * head_dim if kt is None else kt
    kh = head_dim if kh is None else kh
    return lib.qgemv_kv_read(cache("f16", kv_heads, head_dim), 64, 4, 2, None, 64, n, 1, 256, kt, kh, 1 << 20,
                             kv_heads * head_dim, head_dim, None)

def answer(x):
    print("ANSWER " + json.dumps(x))
"""


def run(code, tmp_path):
    """What `code` (which calls answer(...) once) answers."""
    build.build()
    so = os.path.join(str(tmp_path), "fake_cuda_runtime.so")
    if not os.path.exists(so):
        subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "fake_cuda_runtime.c")], check=True)
    r = subprocess.run([sys.executable, "-c", PRELUDE.format(root=os.path.dirname(HERE)) + code], capture_output=True,
                       text=True, timeout=120, env={**os.environ, "LD_PRELOAD": so})
    assert r.returncode == 0, f"the child ended with {r.returncode}:\n{r.stdout}{r.stderr}"
    return json.loads(r.stdout.split("ANSWER ")[1])
