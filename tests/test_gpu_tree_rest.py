"""Rows that no request owns, cleared by the layout: of a padded batch, behind a
count that is cut, without any owned row, and of a graph that is replayed with
fewer rows than the step before it had."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_tree import _lib, _spx, i32, signed, starts  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("news,pad,max_q", [([1], 0, 1), ([1], 1, 1), ([5, 0, 3], 200, 5), ([0, 0], 7, 1), ([0, 64, 2], 65, 64),
                                            ([9, 4, 12], 3, 6), ([9, 4, 12], 0, 6), ([2, 3], 5, 0), ([1] * 300, 1000, 1)])
def test_rows_of_nobody(news, pad, max_q, chain):
    spx = _spx()
    N = sum(news) + pad
    lens = [t + 3 * b for b, t in enumerate(news)]
    parents = [[-1] + [i // 2 for i in range(t - 1)] if t else [] for t in news]
    if chain:
        parents = [[i - 1 for i in range(t)] for t in news]
    flat = i32([p for par in parents for p in par] + [0] * pad)
    guard = 16
    bufs = {n: torch.full((N + 2 * guard,), 77, dtype=torch.int64 if n == "mask" else torch.int32, device="cuda")
            for n in ("req", "slot", "pos", "mask")}
    outs = {n: x[guard:guard + N] for n, x in bufs.items()}
    args, keep = spx.tree_layout_args(starts(news), i32(lens), max_q, parent=None if chain else flat, clear_rest=True, **outs)
    spx.spx_tree_layout(args)
    want = {"req": [], "slot": [], "pos": [], "mask": []}
    for b, (t, n, par) in enumerate(zip(news, lens, parents)):
        T, seen = min(t, max_q), []
        for i in range(t):
            p = par[i]
            seen.append((seen[p] if 0 <= p < i else 0) | 1 << i)
            own = i < T
            want["req"].append(b if own else -1)
            want["slot"].append(n - T + i if own else -1)
            want["pos"].append(n - T + bin(seen[-1]).count("1") - 1 if own else -1)
            want["mask"].append(signed(seen[-1]) if own else 0)
    for n, x in bufs.items():
        rest = 0 if n == "mask" else -1
        assert x.tolist() == [77] * guard + want[n] + [rest] * pad + [77] * guard, n


def test_rows_of_nobody_of_long_chains():
    spx = _spx()
    news, pad = [200, 0, 65, 4097], 500
    N = sum(news) + pad
    req, slot, pos = (torch.full((N,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
    args, keep = spx.tree_layout_args(starts(news), i32([n + 1 for n in news]), 4000, req=req, slot=slot, pos=pos, clear_rest=True)
    spx.spx_tree_layout(args)
    own = [min(n, 4000) for n in news]
    want = [x for b, (n, t) in enumerate(zip(news, own)) for x in [b] * t + [-1] * (n - t)] + [-1] * pad
    at = [x for n, t in zip(news, own) for x in [n + 1 - t + i for i in range(t)] + [-1] * (n - t)] + [-1] * pad
    assert req.tolist() == want and slot.tolist() == at and pos.tolist() == at


@pytest.mark.parametrize("q_start", [[-5, 10 ** 9, 3], [10 ** 9, -5, 2], [3, 1, 0], [-2 ** 31, 2 ** 31 - 1, -2 ** 31], [0, 0, 0],
                                     [2 ** 31 - 1] * 3])
def test_starts_that_do_not_ascend_stay_in_bounds(q_start):
    spx = _spx()
    N, guard = 40, 64
    bufs = [torch.full((N + 2 * guard,), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
    mask = torch.full((N + 2 * guard,), 77, dtype=torch.int64, device="cuda")
    req, slot, pos = (x[guard:guard + N] for x in bufs)
    args, keep = spx.tree_layout_args(i32(q_start), i32([9, 9]), 30, req=req, slot=slot, pos=pos, mask=mask[guard:guard + N],
                                      clear_rest=True)
    spx.spx_tree_layout(args)
    for x in bufs + [mask]:
        assert (x[:guard] == 77).all() and (x[guard + N:] == 77).all()


def test_a_replay_with_fewer_rows_leaves_accepted_tokens_alone():
    """Layout and append in one graph: a step of 8 and 8 rows, of which 3 and 1 are kept, then one of 2 and 3 rows.  The
    rows behind them still hold the keys of the first step's rows, for places that are accepted tokens' by now."""
    spx = _spx()
    torch.manual_seed(0)
    N, kv, D, page = 16, 2, 64, 16
    k, v = (torch.zeros(6, page, kv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    table, lens, q_start = i32([[0, 1, 2], [3, 4, 5]]), i32([20 + 8, 9 + 8]), i32([0, 8, 16])
    cache = spx.KvCache(k, v, table, lens)
    rows = torch.randn(N, 2 * kv, D, device="cuda").half()
    parent = i32([-1, 0, 0, 1, 1, 2, 2, 3] * 2)
    req, slot, pos = (torch.full((N,), -1, dtype=torch.int32, device="cuda") for _ in range(3))
    layout, keep = spx.tree_layout_args(q_start, lens, 8, parent=parent, req=req, slot=slot, pos=pos, clear_rest=True)
    append, keep2 = spx.kv_append_args(cache, rows[:, :kv], rows[:, kv:], req, slot, pos=pos)
    spx.spx_tree_layout(layout)  # (loaded before the capture)
    spx.spx_kv_append(append)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spx.spx_tree_layout(layout)
        spx.spx_kv_append(append)
    graph.replay()
    before_k, before_v, first = k.clone(), v.clone(), rows.clone()
    assert torch.equal(k[1, 4:12], first[:8, :kv]) and torch.equal(k[3, 9:16], first[8:15, :kv])
    rows.copy_(torch.randn(N, 2 * kv, D, device="cuda").half())
    lens.copy_(i32([20 + 3 + 2, 9 + 1 + 3]))
    q_start.copy_(i32([0, 2, 5]))
    graph.replay()
    for i, (p, t) in enumerate([(1, 7), (1, 8), (3, 10), (3, 11), (3, 12)]):
        before_k[p, t], before_v[p, t] = rows[i, :kv], rows[i, kv:]
    assert torch.equal(k, before_k) and torch.equal(v, before_v)
    assert req[5:].tolist() == [-1] * 11
