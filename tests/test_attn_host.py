"""The host's side of the cache and attention calls -- choices of kernels, per-device state -- on a stand-in for the CUDA
runtime that executes nothing (no GPU needed)."""
import pytest

import host_choice


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("fake")
    return lambda code: host_choice.run(code, tmp)


@pytest.mark.parametrize("fmt", ["f16", "int8", "q4_0"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_hint_has_a_kernel(host, fmt, d):
    """max_ctx and max_new only guide the choice: 0 and the largest values of either are calls like others, and one token is
    the least that a call has."""
    got = host(f"""
out = {{}}
for ctx in (0, 1, 5000, (1 << 30) - 1, 1 << 30, (1 << 63) - 1):
    for new in (0, 1, 2, 9, 64, 65, 1 << 30, (1 << 63) - 1):
        rc = tree({fmt!r}, head_dim={d}, max_ctx=ctx, max_new=new)
        out[f"{{ctx}} {{new}}"] = [rc, [n[-1] for n in notes() if n[0] == "launch"]]
answer(out)
""")
    assert len(got) == 48
    for hint, (rc, kernels) in got.items():
        assert rc == 0 and kernels, hint
        ctx, new = map(int, hint.split())
        # contexts bounded by more than 768 positions are split, and joined
        assert ("join" in kernels[-1]) == (ctx + new > 768), (hint, kernels)
    for ctx in (0, 5000):
        assert got[f"{ctx} 0"] == got[f"{ctx} 1"]
