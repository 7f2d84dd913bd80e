"""Waits of the key/value attention launch for many rows that run out where a
block has many units of a tile or two, so that its ring of copies goes round while
copies are under way: what gave up hands no slot on, the call returns, and the
workspace serves again once it is initialised."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, _lib, _spx, call, make, mask_tensor  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# (units of one tile: 12 to 40 a block; of two; two tiles of rows a unit, on one key tile and on several)
SHAPES = [([100] * 120, [17] * 120, 16, 16, 128, True, F16), ([128] * 300, [64] * 300, 8, 8, 64, True, BF16),
          ([200] * 150, [33] * 150, 16, 16, 128, False, BF16), ([130] * 300, [130] * 300, 8, 8, 64, False, F16),
          ([700, 260] * 60, [300, 140] * 60, 8, 4, 128, False, BF16)]


def give_up(s, ws, want, limit, times):
    """Calls with that limit; how many of them report that a wait ran out."""
    spx, ran_out = _spx(), 0
    for _ in range(times):
        out = torch.zeros_like(want)
        args, keep = spx.kv_attention_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                           tree=mask_tensor(s), wait_budget_ns=limit)
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
    return ran_out


@pytest.mark.parametrize("lens,news,heads,kv,D,tree,dtype", SHAPES)
@pytest.mark.parametrize("limit", [1, 700, 5000])
def test_blocks_with_many_units(lens, news, heads, kv, D, tree, dtype, limit):
    s = make(lens, news, heads=heads, kv=kv, D=D, dtype=dtype, tree=tree)
    want, _ = call(s)
    ws = _spx().new_kv_workspace(s["q"], s["cache"], s["max_q"], s["max_len"])
    print("ran out", give_up(s, ws, want, limit, 4))


@pytest.mark.parametrize("lens,news,heads,kv,D,tree,dtype", SHAPES + [
    ([200], [20], 8, 4, 128, True, F16), ([9000, 40, 700], [64, 40, 9], 8, 2, 128, True, F16),
    ([3000] * 8, [33] * 8, 16, 16, 64, False, BF16), ([900], [700], 4, 4, 128, False, F16),
    ([4000, 300], [1500, 200], 8, 2, 64, False, BF16), ([1], [1], 24, 1, 128, True, F16)])
def test_a_limit_below_a_microsecond_runs_out(lens, news, heads, kv, D, tree, dtype):
    """No unit is described within a nanosecond: every call has a wait that runs out, and says so."""
    s = make(lens, news, heads=heads, kv=kv, D=D, dtype=dtype, tree=tree)
    want, _ = call(s)
    ws = _spx().new_kv_workspace(s["q"], s["cache"], s["max_q"], s["max_len"])
    assert give_up(s, ws, want, 1, 5) == 5
