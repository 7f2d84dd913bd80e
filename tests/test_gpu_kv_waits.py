"""Waits of the key/value attention launch for many rows: none runs out while
another stream keeps the SMs busy, and one that does is reported and leaves a
workspace that serves again."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, _lib, call, check, make, mask_tensor  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,news,heads,kv,dtype,tree", [
    ([128 * t + 1 + 17 for t in range(1, 30)], [17] * 29, 16, 16, F16, True), ([300, 129, 1000] * 8, [64] * 24, 8, 2, BF16, True),
    ([4113], [40], 32, 8, F16, False), ([1500, 700], [700, 513], 8, 2, BF16, False)])
def test_no_wait_runs_out(lens, news, heads, kv, dtype, tree):
    s = make(lens, news, heads=heads, kv=kv, dtype=dtype, tree=tree)
    first, lse = call(s)
    check(s, first, lse)
    other, noise = torch.cuda.Stream(), torch.randn(1 << 22, device="cuda")
    for _ in range(60):
        with torch.cuda.stream(other):
            for _ in range(4):
                noise.mul_(1.0001).sin_()
        # (call() asserts that the workspace's status is clean)
        assert torch.equal(call(s, wait_budget_ns=1_000_000_000)[0], first)


@pytest.mark.parametrize("lens,news,heads,kv,tree", [([200], [20], 8, 4, True), ([9000, 40, 700], [64, 40, 9], 8, 2, True),
                                                     ([3000] * 8, [33] * 8, 16, 16, False), ([900], [700], 4, 4, False),
                                                     ([4000, 300], [1500, 200], 8, 2, False)])
def test_a_wait_that_runs_out_is_reported(lens, news, heads, kv, tree):
    """A limit too short for the data to arrive: the call returns, its workspace's status says that a wait ran out (or,
    where everything was there before a suspended wait woke, that nothing did, and the results are right), and the
    workspace serves again once it is initialised."""
    from quantized_expert_gb300 import spx
    s = make(lens, news, heads=heads, kv=kv, tree=tree)
    want, _ = call(s)
    ws = spx.new_kv_workspace(s["q"], s["cache"], s["max_q"], s["max_len"])
    ran_out = 0
    for _ in range(5):
        out = torch.zeros_like(want)
        args, keep = spx.kv_attention_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                           tree=mask_tensor(s), wait_budget_ns=1)
        spx.spx_kv_attention(args)
        torch.cuda.synchronize()
        status = spx.spx_workspace_status(ws)
        assert status in (spx.SPX_OK, spx.SPX_ERR_TIMEOUT)
        if status == spx.SPX_OK:
            assert torch.equal(out, want)
            continue
        ran_out += 1
        ws[:spx.SPX_KV_WORKSPACE_ZERO] = 0
        assert torch.equal(call(s, ws=ws)[0], want)
    print("ran out", ran_out)


def test_results_do_not_depend_on_what_ran_before():
    """Calls of different sizes and inputs in turn, in a stream without waits between: the same bits every time."""
    from quantized_expert_gb300 import spx
    states = [make([2000] * 6, [64] * 6, heads=16, kv=16, dtype=BF16, tree=True, seed=1),
              make([2000] * 6, [64] * 6, heads=16, kv=16, dtype=BF16, tree=True, seed=2),
              make([900, 3000], [17, 17], heads=16, kv=16, dtype=BF16, tree=True, seed=3),
              make([700], [300], heads=8, kv=2, dtype=BF16, seed=4), make([5000] * 3, [1] * 3, heads=8, kv=2, dtype=BF16, seed=5)]
    want, calls = [], []
    for s in states:
        want.append(call(s)[0])
        out = torch.zeros_like(s["q"])
        ws = spx.new_kv_workspace(s["q"], s["cache"], s["max_q"], s["max_len"])
        args, keep = spx.kv_attention_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                           tree=mask_tensor(s))
        calls.append((args, keep, out, ws))
    for i in range(300):
        for args, keep, out, ws in calls:
            spx.spx_kv_attention(args)
        if i % 100 == 99:
            torch.cuda.synchronize()
            for (args, keep, out, ws), w in zip(calls, want):
                assert torch.equal(out, w) and spx.spx_workspace_status(ws) == 0
                out.zero_()
