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


CALLS = {"tree narrow": ("tree('int8', max_new=2)", "tree_kernel"), "tree wide": ("tree('f16', max_new=60)", "tree_wide_kernel"),
         "prompt": ("prompt(n_q=65536, n_k=65536)", "prompt_kernel"), "prompt by runs": ("prompt(n_seqs=2, n_q=600, n_k=12600)", "prompt_kernel")}


@pytest.mark.parametrize("name", list(CALLS))
def test_devices_are_set_up_each(host, name):
    """The limit of shared memory is set on every device, once, and the grid is of the device's own SMs (152 and 100)."""
    call, kernel = CALLS[name]
    got = host(f"""
out = []
for dev in (0, 1, 0, 1):
    fake.fake_set_device(dev)
    out.append([{call}, notes()])
answer(out)
""")
    for k, (rc, notes) in enumerate(got):
        dev = k % 2
        assert rc == 0
        sets = [n for n in notes if n[0] == "attribute"]
        assert [n[1] for n in sets] == [str(dev)] * (k < 2), "set on the device, the first time"
        main = next(n for n in notes if n[0] == "launch" and kernel in n[-1])
        sms = (152, 100)[dev]
        assert main[1] == str(dev) and int(main[2]) in (sms, 2 * sms)
        if k < 2:
            assert int(main[4]) == int(sets[0][3]) > 48 * 1024


@pytest.mark.parametrize("name", list(CALLS))
def test_a_failed_set_up_is_tried_again(host, name):
    call, kernel = CALLS[name]
    fails = ["attributes"] if "tree" in name else ["entry_points", "attributes"]
    got = host(f"""
out = []
for kind in {fails}:
    getattr(fake, "fake_fail_" + kind)(1)
    out.append({call})
notes()
answer([out, {call}, notes()])
""")
    assert got[0] == [3] * len(fails)  # QGEMV_ERR_CUDA
    assert got[1] == 0 and any(n[0] == "launch" and kernel in n[-1] for n in got[2])


@pytest.mark.parametrize("n, heads, ts, hs, apart", [
    (5, 8, 1024, 128, True),          # rows of one tensor
    (5, 8, 128, 640, True),           # head-major
    (5, 8, 128, 128, False),          # every row of a head but the first is the next head's
    (5, 8, 512, 128, False),          # tokens closer than their heads
    (5, 2, 256, 128, True),
    (5, 2, 256, 384, True),           # heads between the tokens of others
    (5, 2, 256, 512, False),
    (2, 2, 256, 512, True),           # that token is not there
    (5, 2, 256, 448, False),          # half of a row
    (1, 8, 128, 128, True),           # one token: its stride means nothing
    (5, 1, 128, 128, True),           # one head
    (1 << 30, 2, 128, 1 << 37, True),
    (1 << 30, 2, 128, (1 << 37) - 128, False),
    (1 << 30, 2, 1 << 38, (1 << 38) - 1024, True),
    (1 << 30, 3, 1 << 38, 1 << 37, False),
])
def test_overlapping_outputs_are_refused(host, n, heads, ts, hs, apart):
    """Two rows of an output that share an element would be written by blocks that know nothing of one another."""
    got = host(f"""
out = [read(kv_heads={heads}, n={n}, kt={ts}, kh={hs})]
if {n} < 1 << 20:
    out += [tree("f16", kv_heads={heads}, q_heads={heads}, n={n}, ot={ts}, oh={hs}),
            prompt(kv_heads={heads}, q_heads={heads}, n_q={n}, n_k={n}, ot={ts}, oh={hs})]
answer(out)
""")
    assert got == [0 if apart else 1] * len(got)  # QGEMV_OK, QGEMV_ERR_ARG
