"""GPU test of the thin bindings of the cache and attention calls, which take addresses: they and the torch-level calls give the
same bits."""
import pytest

from bit_weight_only_gb300 import build, qgemv

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]


def test_bindings_agree_with_the_torch_level_calls():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    qgemv.load()
    n, hq, hkv, d = 70, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, cu, ctx, cu_q = i32([list(range(5))]), i32([0, n]), i32([n - 3]), i32([0, 3])
    slots = torch.arange(n, device="cuda")
    ws = qgemv.AttnWorkspace(1, hq, d)
    caches = [qgemv.KVCache("int8", 5, 16, hkv, d) for _ in range(2)]
    s = torch.cuda.current_stream()
    kv = (hkv * d, d)
    caches[0].write(k, v, slots)
    caches[1].pages.zero_()
    qgemv.qgemv_kv_write(caches[1].desc, qgemv.DT_F16, k.data_ptr(), *kv, v.data_ptr(), *kv, slots.data_ptr(), n, s)
    want = caches[0].read(table, None, cu, n)
    got = tuple(torch.empty_like(t) for t in want)
    qgemv.qgemv_kv_read(caches[1].desc, table.data_ptr(), 5, 1, None, cu.data_ptr(), n, qgemv.DT_F16, got[0].data_ptr(), *kv,
                        got[1].data_ptr(), *kv, s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want, lse = caches[0].attend(q[:3], table, ctx, cu_q, max_ctx=n, max_new=3, workspace=ws)
    out, lse2 = torch.empty_like(want), torch.empty_like(lse)
    qgemv.qgemv_attn_tree(caches[1].desc, table.data_ptr(), 5, 1, ctx.data_ptr(), q.data_ptr(), hq * d, d, hq, cu_q.data_ptr(),
                          3, None, n, 3, d ** -0.5, out.data_ptr(), hq * d, d, lse2.data_ptr(), ws.ptr, ws.nbytes, s)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    want, lse = qgemv.attn_prompt(q, k, v, cu, cu, max_q=n, workspace=ws)
    out, lse2 = torch.empty_like(want), torch.empty_like(lse)
    qgemv.qgemv_attn_ws_init(ws.ptr, ws.nbytes, s)
    qgemv.qgemv_attn_prompt(qgemv.DT_F16, d, hq, hkv, q.data_ptr(), hq * d, d, k.data_ptr(), *kv, v.data_ptr(), *kv, 1,
                            cu.data_ptr(), cu.data_ptr(), n, n, n, d ** -0.5, out.data_ptr(), hq * d, d, lse2.data_ptr(),
                            ws.ptr, ws.nbytes, s)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    assert qgemv.qgemv_attn_status(ws.ptr) == qgemv.QGEMV_OK
