"""Trees of drafted tokens: their layout and their acceptance against a walk on
the host, and a whole step of several requests through the four calls."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from quantized_expert_gb300 import build, spx
    build.build()
    spx.load()
    yield


def _spx():
    from quantized_expert_gb300 import spx
    return spx


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(news):
    return i32([sum(news[:b]) for b in range(len(news) + 1)])


def signed(m):
    return m - (1 << 64) if m >> 63 else m


def run_layout(news, lens, parents, pad=3, chain=False, max_q=None, mask=True):
    spx = _spx()
    N = sum(news) + pad
    flat = None if chain else i32([p for par in parents for p in par] + [0] * pad)
    req, slot, pos = (torch.full((N,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
    m = torch.full((N,), 77, dtype=torch.int64, device="cuda") if mask else None
    args, keep = spx.tree_layout_args(starts(news), i32(lens), max_q or max(max(news), 1), parent=flat, req=req, slot=slot,
                                      pos=pos, mask=m)
    spx.spx_tree_layout(args)
    want = {"req": [], "slot": [], "pos": [], "mask": []}
    for b, (t, n, par) in enumerate(zip(news, lens, parents)):
        seen = []
        for i, p in enumerate(par):
            seen.append((seen[p] if 0 <= p < i else 0) | 1 << i)
            want["req"].append(b)
            want["slot"].append(n - t + i)
            want["pos"].append(n - t + bin(seen[-1]).count("1") - 1)
            want["mask"].append(signed(seen[-1]) if t <= 64 else 0)
    for name, got in (("req", req), ("slot", slot), ("pos", pos), ("mask", m)):
        if got is not None:
            assert got.tolist() == want[name] + [77] * pad, name


@pytest.mark.parametrize("news", [[1], [2], [64], [63, 0, 1, 33, 32, 31], [17] * 70, [0, 0, 5]])
@pytest.mark.parametrize("shape", ["random", "deep", "flat", "broken"])
def test_layout(news, shape):
    g = random.Random(len(news))
    par = {"random": lambda i: g.randrange(i) if i else -1, "deep": lambda i: i - 1, "flat": lambda i: 0 if i else -1,
           "broken": lambda i: g.choice([i, i + 1, -1, -2 ** 31, 2 ** 31 - 1, i - 1])}[shape]
    run_layout(news, [t + g.randrange(500) for t in news], [[par(i) for i in range(t)] for t in news])


@pytest.mark.parametrize("news", [[1], [200, 0, 64, 65, 4097], [1] * 300])
def test_layout_of_chains(news):
    run_layout(news, [t + 5 * b for b, t in enumerate(news)], [[i - 1 for i in range(t)] for t in news], chain=True,
               mask=max(news) <= 64)


def walk(parent, token, target):
    way = [0] if parent else []
    while way:
        fit = [i for i in range(way[-1] + 1, len(parent)) if parent[i] == way[-1] and token[i] == target[way[-1]]]
        if not fit:
            break
        way.append(fit[0])
    return way


def accept_case(news, lens, layers, kv, D, page, order, dtype, seed, vocab=3, missing=False):
    """Trees with few distinct tokens, so that paths are long; every buffer's values tell where they came from."""
    spx, g = _spx(), random.Random(seed)
    tg = torch.Generator(device="cuda").manual_seed(seed)
    B, N = len(news), sum(news) + 2
    parents = [[-1] + [g.randrange(max(0, i - 3), i) for i in range(1, t)] if t else [] for t in news]
    tokens = [[g.randrange(vocab) for _ in range(t)] for t in news]
    targets = [[g.randrange(vocab) for _ in range(t)] for t in news]
    per = -(-max(max(lens), 1) // page)
    pages = B * per + 2
    shape = {"token": (pages, page, kv, D), "head": (pages, kv, page, D)}[order]
    bufs = [torch.randn(shape, generator=tg, device="cuda").to(dtype) for _ in range(2 * layers)]
    views = [x if order == "token" else x.transpose(1, 2) for x in bufs]
    table = torch.randperm(pages, generator=tg, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    if missing:
        table[0, (lens[0] - 1) // page] = -1
    want = [x.clone() for x in views]
    n_kept, path, nxt, lens_out = [], [], [], []
    tl = table.tolist()
    for b, t in enumerate(news):
        way = walk(parents[b], tokens[b], targets[b])
        n_kept.append(len(way))
        path += way + [-1] * (t - len(way))
        nxt.append(targets[b][way[-1]] if way else -1)
        lens_out.append(lens[b] - t + len(way))
        for d, i in enumerate(way):
            a, z = lens[b] - t + i, lens[b] - t + d
            if tl[b][a // page] >= 0 and tl[b][z // page] >= 0:
                for old, now in zip(views, want):
                    now[tl[b][z // page], z % page] = old[tl[b][a // page], a % page]

    def flat(x):
        return i32([v for r in x for v in r] + [0, 0])

    caches = [spx.KvCache(views[2 * l], views[2 * l + 1], table, i32(lens)) for l in range(layers)]
    for c in caches:
        c.lens = caches[0].lens
    got = dict(n_kept=torch.full((B,), 77, dtype=torch.int32, device="cuda"), lens_out=torch.full((B,), 77, dtype=torch.int32, device="cuda"),
               next_token=torch.full((B,), 77, dtype=torch.int32, device="cuda"), path=torch.full((N,), 77, dtype=torch.int32, device="cuda"))
    args, keep = spx.tree_accept_args(caches, starts(news), max(max(news), 1), flat(parents), flat(tokens), flat(targets), **got)
    spx.spx_tree_accept(args)
    assert got["n_kept"].tolist() == n_kept and got["next_token"].tolist() == nxt
    assert got["lens_out"].tolist() == lens_out and got["path"].tolist() == path + [77, 77]
    for now, x in zip(want, views):
        assert torch.equal(now, x)
    return n_kept


@pytest.mark.parametrize("news,lens", [([1], [1]), ([64], [64]), ([17], [500]), ([64, 0, 1, 33, 5], [100, 9, 1, 300, 77]),
                                       ([8] * 40, [40] * 40)])
@pytest.mark.parametrize("layers,kv,D,page,order,dtype", [
    (1, 1, 64, 16, "token", torch.float16), (3, 5, 128, 48, "head", torch.bfloat16), (40, 2, 64, 64, "token", torch.bfloat16)])
@pytest.mark.parametrize("vocab", [1, 2, 1000])
def test_accept(news, lens, layers, kv, D, page, order, dtype, vocab):
    kept = accept_case(news, lens, layers, kv, D, page, order, dtype, seed=layers, vocab=vocab)
    if vocab == 1:  # every token is the target's: a leaf is reached
        assert max(kept) > 1 or max(news) == 1


def test_accept_with_a_missing_page():
    accept_case([30, 30], [40, 40], 2, 2, 64, 16, "token", torch.float16, seed=1, vocab=1, missing=True)


def test_accept_of_a_chain_moves_nothing():
    spx = _spx()
    k, v = (torch.randn(4, 16, 2, 64, device="cuda").half() for _ in range(2))
    cache = spx.KvCache(k, v, i32([[1, 2, 3]]), i32([40]))
    was = k.clone()
    out = [torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(3)]
    path = torch.empty(6, dtype=torch.int32, device="cuda")
    args, keep = spx.tree_accept_args([cache], i32([0, 6]), 6, i32([-1, 0, 1, 2, 3, 4]), i32([9, 1, 2, 3, 4, 5]),
                                      i32([1, 2, 3, 8, 5, 6]), out[0], path, out[1], out[2])
    spx.spx_tree_accept(args)
    assert path.tolist() == [0, 1, 2, 3, -1, -1] and [x.item() for x in out] == [4, 8, 38] and torch.equal(k, was)


def test_accept_without_caches_to_move():
    from quantized_expert_gb300 import spx
    import ctypes as C
    k = torch.empty(4, 16, 2, 64, device="cuda", dtype=torch.float16)
    cache = spx.KvCache(k, k.clone(), i32([[1, 2, 3]]), i32([40]))
    out = torch.empty(3, dtype=torch.int32, device="cuda")
    path = torch.empty(3, dtype=torch.int32, device="cuda")
    args, keep = spx.tree_accept_args([cache], i32([0, 3]), 3, i32([-1, 0, 0]), i32([9, 1, 2]), i32([2, 2, 5]), out[0:1], path,
                                      out[1:2], out[2:3])
    args.n_layers, args.layer_k, args.layer_v = 0, None, None
    spx.spx_tree_accept(args)
    assert path.tolist() == [0, 2, -1] and out.tolist() == [2, 5, 39]


def test_a_step_of_trees():
    """Layout, append, attention and acceptance in one graph, against a model that ran the accepted tokens one after the
    other: the caches and the next step's outputs agree."""
    spx = _spx()
    torch.manual_seed(0)
    H, heads, kv, D, page, B, T, dt = 256, 8, 2, 64, 16, 3, 21, torch.float16
    w = (torch.randn((heads + 2 * kv) * D, H, device="cuda") * H ** -0.5).to(dt)
    embed = torch.randn(50, H, device="cuda").to(dt)
    unembed = torch.randn(50, heads * D, device="cuda").to(dt)
    angle = torch.arange(256, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    cos, sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()
    norm = torch.ones(D, dtype=dt, device="cuda")
    prompts = [torch.randint(0, 50, (n,), device="cuda") for n in (70, 33, 5)]

    def fresh():
        k, v = (torch.full((40, page, kv, D), math.nan, dtype=dt, device="cuda") for _ in range(2))
        return spx.KvCache(k, v, torch.arange(36, device="cuda").to(torch.int32).reshape(3, 12), i32([0, 0, 0]))

    def attend(cache, x, news, max_q, max_len, ws, parent, bufs):
        """One layer's step on rows x; the caches' lengths count the new rows."""
        N = x.shape[0]
        qkv = (x @ w.T).view(N, heads + 2 * kv, D)
        args, keep = spx.tree_layout_args(news, cache.lens, max_q, parent=parent, req=bufs["req"], slot=bufs["slot"],
                                          pos=bufs["pos"], mask=bufs["mask"] if parent is not None else None)
        spx.spx_tree_layout(args)
        q = torch.empty(N, heads, D, dtype=dt, device="cuda")
        a2, keep2 = spx.kv_append_args(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], bufs["req"], bufs["slot"],
                                       pos=bufs["pos"], q=qkv[:, :heads], q_out=q, q_norm=norm, k_norm=norm, cos=cos, sin=sin)
        spx.spx_kv_append(a2)
        out = torch.empty_like(q)
        a3, keep3 = spx.kv_attention_args(q, cache, news, max_q, max_len, D ** -0.5, out, ws,
                                          tree=bufs["mask"] if parent is not None else None)
        spx.spx_kv_attention(a3)
        return out, [args, keep, a2, keep2, a3, keep3, qkv, q]

    def bufs(N):
        return dict(req=torch.empty(N, dtype=torch.int32, device="cuda"), slot=torch.empty(N, dtype=torch.int32, device="cuda"),
                    pos=torch.empty(N, dtype=torch.int32, device="cuda"), mask=torch.zeros(N, dtype=torch.int64, device="cuda"))

    def prompt(cache, seqs):
        news = [len(x) for x in seqs]
        cache.lens.add_(i32(news))
        x = embed[torch.cat(seqs)]
        ws = spx.new_kv_workspace(torch.empty(len(x), heads, D, dtype=dt, device="cuda"), cache, max(news), 190)
        out, keep = attend(cache, x, starts(news), max(news), 190, ws, None, bufs(len(x)))
        torch.cuda.synchronize()
        return out

    cache = fresh()
    prompt(cache, prompts)
    base = [len(x) for x in prompts]
    # the tree: random parents; tokens are drafted so that the target agrees along some paths
    g = random.Random(2)
    parents = [[-1] + [g.randrange(max(0, i - 5), i) for i in range(1, T)] for _ in range(B)]
    tokens = torch.randint(0, 50, (B, T), device="cuda")
    for b in range(B):  # (a target that depends on the token alone makes agreement likely: the row's best by itself)
        for i in range(1, T):
            if g.random() < 0.7:
                tokens[b, i] = (tokens[b, parents[b][i]] * 7 + 3) % 50
    target = (tokens * 7 + 3) % 50
    parent = i32([p for par in parents for p in par])
    token, target = tokens.flatten().to(torch.int32).contiguous(), target.flatten().to(torch.int32).contiguous()
    x = embed[token.long()]
    news = starts([T] * B)
    ws = spx.new_kv_workspace(torch.empty(B * T, heads, D, dtype=dt, device="cuda"), cache, T, 190)
    n_kept, nxt, lens_out = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
    path, room = torch.empty(B * T, dtype=torch.int32, device="cuda"), bufs(B * T)
    args, keep = spx.tree_accept_args([cache], news, T, parent, token, target, n_kept, path, nxt, lens_out)
    x @ w.T  # (the library's handles exist before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.lens.add_(T)
        out, kept_alive = attend(cache, x, news, T, 190, ws, parent, room)
        spx.spx_tree_accept(args)
        cache.lens.copy_(lens_out)
    graph.replay()
    torch.cuda.synchronize()
    kept = n_kept.tolist()
    assert max(kept) > 2 and cache.lens.tolist() == [a + c for a, c in zip(base, kept)]
    # the same tokens in a row
    other = fresh()
    prompt(other, prompts)
    seqs, rows = [], []
    for b in range(B):
        way = path[b * T:b * T + kept[b]].tolist()
        assert nxt[b].item() == target[b * T + way[-1]].item()
        seqs.append(tokens[b, way])
        rows += [b * T + i for i in way]
    straight = prompt(other, seqs)
    # (products of other shapes: fp16 roundings of x W and what attention makes of them)
    assert (straight.double() - out[rows].double()).norm() <= 8 * 2.0 ** -11 * straight.double().norm()
    for b in range(B):
        n = base[b] + kept[b]
        at = torch.arange(n, device="cuda")
        for mine, his in ((cache.k, other.k), (cache.v, other.v)):
            a, c = (y[cache.block_table[b, at // page].long(), at % page].double() for y in (mine, his))
            assert (a - c).norm() <= 4 * 2.0 ** -11 * c.norm()
