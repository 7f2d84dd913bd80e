"""Acceptance with block-table entries that name no page: a row of the path
without one is moved as the zeros that attention reads there, and what has no
page to go to goes nowhere."""
import random

import pytest

torch = pytest.importorskip("torch")

from test_gpu_tree import _lib, _spx, i32, starts, walk  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, -2 ** 31, 10 ** 6])
@pytest.mark.parametrize("order,dtype,layers", [("token", torch.float16, 1), ("head", torch.bfloat16, 33)])
@pytest.mark.parametrize("missing", ["sources", "destinations", "both", "all", "past the table"])
def test_accepted_rows_without_a_page(missing, order, dtype, layers, entry):
    spx, g = _spx(), random.Random(7)
    tg = torch.Generator(device="cuda").manual_seed(7)
    kv, D, page, base, T, B = 3, 64, 16, 10, 64, 3
    per, news, lens = 5, [T] * 3, [base + T] * 3
    pages = B * per + 1
    shape = (pages, page, kv, D) if order == "token" else (pages, kv, page, D)
    bufs = [torch.randn(shape, generator=tg, device="cuda").to(dtype) for _ in range(2 * layers)]
    views = [x if order == "token" else x.transpose(1, 2) for x in bufs]
    table = torch.randperm(pages, generator=tg, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    # paths of 24 rows over all pages of the tree's rows, no other row behind any
    parents = [[-1] * T for _ in range(B)]
    for par in parents:
        way = [0] + sorted(g.sample(range(1, T), 23))
        for a, b in zip(way, way[1:]):
            par[b] = a
    if missing == "past the table":
        table = table[:, :3].contiguous()
    gone = {"sources": [3, 4], "destinations": [1], "both": [0, 2], "all": [0, 1, 2, 3, 4], "past the table": []}[missing]
    for p in gone:
        table[1:, p] = entry
    tl, want = table.tolist(), [x.clone() for x in views]
    kinds = set()
    paths = [walk(par, [0] * T, [0] * T) for par in parents]
    assert all(len(w) == 24 for w in paths)
    for b, way in enumerate(paths):
        for d, i in enumerate(way):
            a, z = base + i, base + d
            have = [x // page < len(tl[b]) and 0 <= tl[b][x // page] < pages for x in (a, z)]
            kinds.add((i != d, *have))
            if i == d or not have[1]:
                continue
            for old, now in zip(views, want):
                now[tl[b][z // page], z % page] = old[tl[b][a // page], a % page] if have[0] else 0
    if missing in ("sources", "both", "past the table"):
        assert (True, False, True) in kinds
    caches = [spx.KvCache(views[2 * l], views[2 * l + 1], table, i32(lens)) for l in range(layers)]
    for c in caches:
        c.lens = caches[0].lens
    n_kept, nxt, lens_out = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
    path = torch.empty(B * T, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B * T, dtype=torch.int32, device="cuda")
    args, keep = spx.tree_accept_args(caches, starts(news), T, i32([p for par in parents for p in par]), zero, zero.clone(), n_kept,
                                      path, nxt, lens_out)
    spx.spx_tree_accept(args)
    assert n_kept.tolist() == [len(w) for w in paths] and lens_out.tolist() == [base + len(w) for w in paths]
    for now, x in zip(want, views):
        assert torch.equal(now, x)
