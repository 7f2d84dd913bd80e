"""Speculation with trees of drafted tokens over an ordinary paged cache of keys
and values, as measurable operators:

* ``tree_layout``: from the parents of the drafted rows, which rows each sees,
  where each is cached and at which position it is rotated;
* ``kv_append``: the new tokens' keys (and queries) normalised per head and
  rotated, keys and values written to the cache;
* ``kv_attention``: attention of the new tokens (one, a tree, a prompt's chunk)
  over the cache, query heads in groups that share a key head;
* ``tree_accept``: the longest path of drafted tokens that the target agrees
  with, and its keys and values moved together in every layer's cache.

``own`` selects between the plain form (elementary torch operations in 32
bits) and the library's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
VOCAB = 32000
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the draft step of one request early in its answer, a key head for every query head: launch latency
        dict(name="decode_short", op="attention", dtype="f16", heads=16, kv=16, dim=128, batch=1, tokens=1, context=517,
             ragged=False, tree=False, page=64, order="token", pad=0),
        # the draft step of one request behind a long document, four query heads a key head: cache bandwidth
        dict(name="decode_long", op="attention", dtype="f16", heads=32, kv=8, dim=128, batch=1, tokens=1, context=65536,
             ragged=False, tree=False, page=64, order="token", pad=0),
        # draft steps of many requests of different lengths, pages with a head's tokens together
        dict(name="decode_batch", op="attention", dtype="bf16", heads=16, kv=16, dim=128, batch=32, tokens=1,
             context=4096, ragged=True, tree=False, page=32, order="head", pad=0),
        # the verify pass of one request: the last token and a tree of 16 drafted ones
        dict(name="tree_one", op="attention", dtype="f16", heads=32, kv=8, dim=128, batch=1, tokens=17, context=4113,
             ragged=False, tree=True, page=64, order="token", pad=0),
        # verify passes of several requests with wide trees, rows of a padded batch behind them
        dict(name="tree_batch", op="attention", dtype="bf16", heads=16, kv=16, dim=128, batch=16, tokens=64,
             context=3001, ragged=True, tree=True, page=64, order="token", pad=5),
        # prompt chunks of several requests behind cached text, odd sizes, the smallest pages
        dict(name="prompt_chunks", op="attention", dtype="bf16", heads=32, kv=8, dim=128, batch=4, tokens=1021,
             context=6007, ragged=True, tree=False, page=16, order="token", pad=0),
        # the new tokens of one verify pass go to the cache of one layer
        dict(name="append_tree", op="append", dtype="f16", heads=32, kv=8, dim=128, batch=1, tokens=17, context=4113,
             tree=True, page=64, order="token", rotary=128, interleaved=False, norms=False, pad=0),
        # the tokens of prompt chunks, with norms of queries and keys
        dict(name="append_prompt", op="append", dtype="bf16", heads=32, kv=8, dim=128, batch=4, tokens=2048,
             context=8192, tree=False, page=16, order="token", rotary=128, interleaved=False, norms=True, pad=0),
        # the tree of one verify pass laid out: launch latency
        dict(name="layout_one", op="layout", batch=1, tokens=17, context=4113, tree=True, pad=0),
        # the largest trees of many requests
        dict(name="layout_batch", op="layout", batch=64, tokens=64, context=2048, tree=True, pad=0),
        # the end of one verify pass: the path accepted, the caches of 24 layers moved together
        dict(name="accept_one", op="accept", dtype="f16", kv=16, dim=128, batch=1, tokens=17, context=512, layers=24,
             page=64, order="token", pad=0),
        # of several requests with wide trees, 32 layers
        dict(name="accept_batch", op="accept", dtype="bf16", kv=8, dim=128, batch=16, tokens=64, context=256, layers=32,
             page=16, order="token", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = [work(c) for c in listed()]
    limits = {op: [max(w[k] for w, c in zip(top, listed()) if c["op"] == op) for k in ("bytes", "flops")]
              for op in ("attention", "append", "layout", "accept")}
    while True:
        c = dict(op=rng.choice(["attention", "attention", "attention", "append", "layout", "accept"]),
                 batch=_log(rng, 1, 64), pad=rng.choice([0, 0, 1, 7, 64]))
        if c["op"] != "layout":
            c["heads"], c["kv"] = rng.choice([(16, 16), (32, 8), (32, 8), (28, 4), (8, 1), (20, 20), (12, 4), (40, 8),
                                              (64, 8), (24, 1)])
            c.update(dtype=rng.choice(["f16", "bf16"]), dim=rng.choice([64, 128, 128]),
                     page=rng.choice([16, 32, 48, 64, 128]), order=rng.choice(["token", "head"]))
        if c["op"] == "attention":
            c["tree"] = rng.random() < 0.4
            c["tokens"] = rng.randint(2, 64) if c["tree"] else rng.choice([1, rng.randint(2, 33), _log(rng, 34, 4096)])
            c["context"], c["ragged"] = max(_log(rng, 64, 65536), c["tokens"]), rng.random() < 0.6
            if c["batch"] * c["context"] > 1 << 18 or c["batch"] * c["tokens"] * c["context"] * c["heads"] > 1 << 30:
                continue
        elif c["op"] == "append":
            c["tree"] = rng.random() < 0.5
            c["tokens"] = rng.randint(2, 64) if c["tree"] else _log(rng, 1, 4096)
            c["context"] = max(_log(rng, 64, 16384), c["tokens"])
            c.update(rotary=rng.choice([0, c["dim"] // 2, c["dim"], c["dim"]]), interleaved=rng.random() < 0.5,
                     norms=rng.random() < 0.5)
            if c["batch"] * c["context"] > 1 << 16:
                continue
        elif c["op"] == "layout":
            c["tree"] = rng.random() < 0.8
            c["tokens"] = rng.randint(1, 64)
            c["context"] = _log(rng, 64, 65536)
        else:
            c.update(tokens=rng.randint(1, 64), context=_log(rng, 64, 2048), layers=_log(rng, 1, 64))
            if c["batch"] * c["context"] * c["layers"] > 1 << 17:
                continue
        w = work(c)
        if w["bytes"] <= limits[c["op"]][0] and w["flops"] <= limits[c["op"]][1]:
            return c


def _requests(c):
    """Cached length (new tokens included) and new tokens of each request: the
    same for every seed."""
    B, T, L = c["batch"], c["tokens"], c["context"]
    if not c.get("ragged", c["op"] in ("layout", "accept")):
        return [L] * B, [T] * B
    g = random.Random("%s %s %s" % (B, T, L))
    lens = [L] + [g.randint(max(1, L // 8), L) for _ in range(B - 1)]
    news = [T] + [g.randint(max(1, T // 2), T) for _ in range(B - 1)]
    return lens, [min(t, n) for t, n in zip(news, lens)]


def _kept(c):
    """Rows that each request keeps (the last token and what is accepted), at
    most half of a tree, or a chain."""
    g = random.Random("%s %s %s kept" % (c["batch"], c["tokens"], c["context"]))
    return [g.randint(1, (t + 1) // 2) for t in _requests(c)[1]]


def work(c):
    lens, news = _requests(c)
    n = sum(news)
    if c["op"] == "layout":
        return {"bytes": n * (4 + 3 * 4 + 8) + 4 * (2 * c["batch"] + 1), "flops": 2.0 * n}
    e = 2
    if c["op"] == "accept":
        moved = sum(k - 1 for k in _kept(c))
        return {"bytes": moved * c["layers"] * 2 * c["kv"] * c["dim"] * e * 2 + 16 * n + 20 * c["batch"],
                "flops": 2.0 * n}
    if c["op"] == "append":
        rows = min(c["context"], n)
        return {"bytes": n * ((c["heads"] + 2 * c["kv"]) * c["dim"] * e * 2 + 12) + rows * c["rotary"] * 4,
                "flops": n * (c["heads"] + c["kv"]) * (3.0 * c["rotary"] + (4.0 * c["dim"] if c["norms"] else 1.0))}
    pairs = sum(t * (m - t) + t * (t + 1) // 2 for m, t in zip(lens, news))
    return {"bytes": 2 * n * c["heads"] * c["dim"] * e + 2 * sum(lens) * c["kv"] * c["dim"] * e +
            4 * sum(-(-m // c["page"]) for m in lens), "flops": 4.0 * c["heads"] * c["dim"] * pairs}


# ----------------------------------------------------------------- inputs --
def _trees(c, news, rng):
    """Parents of each request's rows (row 0: the last token, the others drafted
    behind an earlier row)."""
    if not c.get("tree", True):
        return [[i - 1 for i in range(t)] for t in news]
    return [[-1] + [rng.randint(max(0, i // 2 - 2), i - 1) for i in range(1, t)] for t in news]


def _masks(parents):
    out = []
    for par in parents:
        seen = []
        for i, p in enumerate(par):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out += [m - (1 << 64) if m >> 63 else m for m in seen]
    return out


def _depths(par):
    d = []
    for p in par:
        d.append(d[p] + 1 if p >= 0 else 0)
    return d


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _layout_lens(c, seed):
    """Cached lengths of a layout case: the seed's own, as a chain's outputs
    follow from them alone."""
    rng = random.Random(seed + 1)
    return [t + rng.randrange(c["context"]) for t in _requests(c)[1]]


def _caches(c, g, dt, layers):
    """Caches whose requests have their pages at random places: keys and values
    [layer][pages][page][kv][dim] (views of pages with a head's tokens together
    where the order is by head), and the block table."""
    per = -(-c["context"] // c["page"])
    pages = per * c["batch"]
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(c["batch"], per).contiguous()
    shape = (pages, c["page"], c["kv"], c["dim"]) if c["order"] == "token" else (pages, c["kv"], c["page"], c["dim"])
    k, v = (torch.randn(layers, *shape, generator=g, device="cuda").to(dt) for _ in range(2))
    return (k, v, table) if c["order"] == "token" else (k.transpose(2, 3), v.transpose(2, 3), table)


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, news = _requests(c)
    B, n = c["batch"], sum(news)
    N = n + c["pad"]
    s = {"case": c, "lens": _i32(lens), "q_start": _i32([0] + [sum(news[:b + 1]) for b in range(B)]),
         "max_q": max(news), "max_len": max(lens), "rows": n}
    parents = _trees(c, news, rng)
    tail = [0] * c["pad"]
    if c["op"] == "layout":
        s["lens"] = _i32(_layout_lens(c, seed))
        s["parent"] = _i32([p for par in parents for p in par] + tail) if c["tree"] else None
        s["req"], s["slot"], s["pos"] = (torch.zeros(N, dtype=torch.int32, device="cuda") for _ in range(3))
        s["mask"] = torch.zeros(N, dtype=torch.int64, device="cuda")
        return s
    dt = DTYPES[c["dtype"]]
    if c["op"] == "accept":
        s["k"], s["v"], s["table"] = _caches(c, g, dt, c["layers"])
        token, target, parent = [], [], []
        for t, kept in zip(news, _kept(c)):
            # the accepted rows lie behind the places they go to (as in a tree written level by level), so that
            # a second pass finds what the first one found
            path = [0] + sorted(rng.sample(range(kept, t), kept - 1))
            par = [-1] + [rng.randint(0, i - 1) for i in range(1, t)]
            for a, b in zip(path, path[1:]):
                par[b] = a
            tgt = [rng.randrange(VOCAB) for _ in range(t)]
            tok = [rng.randrange(VOCAB)] + [tgt[par[i]] if i in path else (tgt[par[i]] + rng.randint(1, 999)) % VOCAB
                                            for i in range(1, t)]
            token, target, parent = token + tok, target + tgt, parent + par
        s["token"], s["target"], s["parent"] = _i32(token + tail), _i32(target + tail), _i32(parent + tail)
        s["n_kept"], s["next"], s["lens_out"] = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        s["path"] = torch.zeros(N, dtype=torch.int32, device="cuda")
        return s
    k, v, s["table"] = _caches(c, g, dt, 1)
    s["k"], s["v"] = k[0], v[0]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    h, kv, d = c["heads"], c["kv"], c["dim"]
    if c["op"] == "append":
        s["qkv"] = normal(N, (h + 2 * kv) * d)  # one projection's output, its parts side by side
        base = [m - t for m, t in zip(lens, news)]
        s["req"] = _i32([b for b, t in enumerate(news) for _ in range(t)] + [-1] * c["pad"])
        s["slot"] = _i32([m + i for m, t in zip(base, news) for i in range(t)] + [-1] * c["pad"])
        s["pos"] = _i32([m + i for m, par in zip(base, parents) for i in _depths(par)] + [-1] * c["pad"])
        if c["norms"]:
            s["q_norm"], s["k_norm"] = ((1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2))
        if c["rotary"]:
            angle = torch.arange(c["context"], device="cuda", dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(0, c["rotary"], 2, device="cuda", dtype=torch.float64) / c["rotary"])
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["q_out"] = torch.zeros(N, h, d, dtype=dt, device="cuda")
        return s
    s["q"] = normal(N, h, d, std=1.5)
    s["scale"] = 1.0 / math.sqrt(d)
    if c["tree"]:
        s["parents"] = parents
        s["mask"] = torch.tensor(_masks(parents) + tail, dtype=torch.int64).cuda()
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(N, h, device="cuda")
    return s


# -------------------------------------------------------------------- run --
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "layout": _own_layout, "accept": _own_accept}[op](state)
    return {"attention": _plain_attention, "append": _plain_append, "layout": _plain_layout,
            "accept": _plain_accept}[op](state)


def _own_attention(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:  # a program keeps its workspace and its argument block from call to call
        cache = spx.KvCache(s["k"], s["v"], s["table"], s["lens"])
        ws = spx.new_kv_workspace(s["q"], cache, s["max_q"], s["max_len"])
        s["call"] = spx.kv_attention_args(s["q"], cache, s["q_start"], s["max_q"], s["max_len"], s["scale"], s["out"],
                                          ws, causal=True, tree=s.get("mask"), lse=s["lse"])
    spx.spx_kv_attention(s["call"][0])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:
        c, N = s["case"], s["qkv"].shape[0]
        q, k, v = (x.view(N, -1, c["dim"]) for x in
                   s["qkv"].split([c["heads"] * c["dim"], c["kv"] * c["dim"], c["kv"] * c["dim"]], -1))
        cache = spx.KvCache(s["k"], s["v"], s["table"], s["lens"])
        s["call"] = spx.kv_append_args(cache, k, v, s["req"], s["slot"], pos=s["pos"], q=q, q_out=s["q_out"],
                                       q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS, cos=s.get("cos"),
                                       sin=s.get("sin"), interleaved=c["interleaved"])
    spx.spx_kv_append(s["call"][0])
    return {"k": s["k"], "v": s["v"], "q": s["q_out"]}


def _own_layout(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:
        s["call"] = spx.tree_layout_args(s["q_start"], s["lens"], s["max_q"], parent=s["parent"], req=s["req"],
                                         slot=s["slot"], pos=s["pos"], mask=s["mask"])
    spx.spx_tree_layout(s["call"][0])
    return {k: s[k] for k in ("req", "slot", "pos", "mask")}


def _own_accept(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:
        caches = [spx.KvCache(k, v, s["table"], s["lens"]) for k, v in zip(s["k"], s["v"])]
        s["call"] = spx.tree_accept_args(caches, s["q_start"], s["max_q"], s["parent"], s["token"], s["target"],
                                         s["n_kept"], s["path"], s["next"], s["lens_out"])
    spx.spx_tree_accept(s["call"][0])
    return {k: s[k] for k in ("n_kept", "path", "next", "lens_out", "k", "v")}


def _padded(s):
    """Row of (request, i) in the batch, cut to the batch; which of them exist;
    the position of the first new token."""
    q_start, lens = s["q_start"].long(), s["lens"].long()
    i = torch.arange(s["max_q"], device="cuda")
    news = q_start[1:] - q_start[:-1]
    return (q_start[:-1, None] + i).clamp(max=s["rows"] - 1), i < news[:, None], lens - news


def _plain_attention(s):
    c = s["case"]
    h, kv, d, T, L = c["heads"], c["kv"], c["dim"], s["max_q"], s["max_len"]
    g, B = h // kv, c["batch"]
    row, new, base = _padded(s)
    at = torch.arange(L, device="cuda")
    page = s["table"].long()[:, at // c["page"]]                              # [B][L]
    k = s["k"][page, at % c["page"]].float().transpose(1, 2)                  # [B][kv][L][d]
    v = s["v"][page, at % c["page"]].float().transpose(1, 2)
    q = s["q"].float()[row].reshape(B, T, kv, g, d).permute(0, 2, 3, 1, 4).reshape(B, kv, g * T, d)
    score = (q @ k.transpose(2, 3) * s["scale"]).reshape(B, kv, g, T, L)
    rel = at - base[:, None]                                                  # [B][L]: index among the new tokens
    if c["tree"]:
        bit = s["mask"][row][:, :, None] >> rel.clamp(0, 63)[:, None] & 1     # [B][T][L]
        seen = (rel < 0)[:, None] | ((bit == 1) & (rel < 64)[:, None])
    else:
        seen = rel[:, None] <= torch.arange(T, device="cuda")[:, None]
    seen = seen & (at < s["lens"].long()[:, None])[:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    m = score.max(-1, keepdim=True).values.clamp(min=-1e30)
    e = torch.exp(score - m)
    z = e.sum(-1, keepdim=True)
    out = ((e / z.clamp(min=1e-30)).reshape(B, kv, g * T, L) @ v).reshape(B, h, T, d)
    lse = (m + torch.log(z)).reshape(B, h, T)
    s["out"][:s["rows"]] = out.permute(0, 2, 1, 3)[new].to(s["q"].dtype)
    s["lse"][:s["rows"]] = lse.permute(0, 2, 1)[new]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_append(s):
    c, n, dt = s["case"], s["rows"], s["qkv"].dtype
    h, kv, d, P = c["heads"], c["kv"], c["dim"], c["rotary"]
    q, k, v = (x.reshape(n, -1, d) for x in s["qkv"][:n].split([h * d, kv * d, kv * d], -1))
    pos = s["pos"][:n].long()

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        if P:
            cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
            if c["interleaved"]:
                a, b = x[..., 0:P:2], x[..., 1:P:2]
                r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = x[..., :P // 2], x[..., P // 2:P]
                r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            x = torch.cat([r, x[..., P:]], -1)
        return x.to(dt)

    slot = s["slot"][:n].long()
    page = s["table"].long()[s["req"][:n].long(), slot // c["page"]]
    s["k"][page, slot % c["page"]] = turned(k, s.get("k_norm"))
    s["v"][page, slot % c["page"]] = v
    s["q_out"][:n] = turned(q, s.get("q_norm"))
    return {"k": s["k"], "v": s["v"], "q": s["q_out"]}


def _plain_layout(s):
    row, new, base = _padded(s)
    B, T = row.shape
    i = torch.arange(T, device="cuda")
    parent = (s["parent"].long()[row] if s["parent"] is not None else i - 1 + 0 * row)
    seen = torch.zeros(B, T, T, dtype=torch.bool, device="cuda")
    for j in range(T):
        p = parent[:, j]
        above = seen.gather(1, p.clamp(min=0)[:, None, None].expand(B, 1, T))[:, 0] & (p >= 0)[:, None]
        seen[:, j] = above | (i == j)
    mask = (seen.long() << i).sum(-1)
    depth = seen.sum(-1) - 1
    n = s["rows"]
    s["req"][:n] = (torch.arange(B, device="cuda")[:, None] + 0 * row)[new].to(torch.int32)
    s["slot"][:n] = (base[:, None] + i)[new].to(torch.int32)
    s["pos"][:n] = (base[:, None] + depth)[new].to(torch.int32)
    s["mask"][:n] = mask[new]
    return {k: s[k] for k in ("req", "slot", "pos", "mask")}


def _plain_accept(s):
    c = s["case"]
    row, new, base = _padded(s)
    B, T = row.shape
    i = torch.arange(T, device="cuda")
    parent, token, target = (s[k].long()[row] for k in ("parent", "token", "target"))
    at = torch.zeros(B, dtype=torch.long, device="cuda")
    alive = torch.ones(B, dtype=torch.bool, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    for d in range(1, T):
        fits = (parent == at[:, None]) & (token == target.gather(1, at[:, None])) & new & (i > 0)
        first = torch.where(fits, i, T).min(-1).values
        alive = alive & (first < T)
        at = torch.where(alive, first, at)
        path[:, d] = torch.where(alive, at, -1)
    kept = (path >= 0).sum(-1)
    s["n_kept"].copy_(kept)
    s["next"].copy_(target.gather(1, at[:, None])[:, 0])
    s["lens_out"].copy_(base + kept)
    s["path"][:s["rows"]] = path[new].to(torch.int32)
    # a row that is not kept stays where it is; one that does not exist stands for the first
    moved = path >= 0
    src = base[:, None] + torch.where(moved, path, torch.where(new, i, 0))
    dst = base[:, None] + torch.where(new, i, 0)
    src_page = s["table"].long().gather(1, src // c["page"])
    dst_page = s["table"].long().gather(1, dst // c["page"])
    for x in (s["k"], s["v"]):
        for layer in x:
            layer[dst_page, dst % c["page"]] = layer[src_page, src % c["page"]]
    return {k: s[k] for k in ("n_kept", "path", "next", "lens_out", "k", "v")}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, request by request."""
    s, c = prepare(case, seed), case
    lens, news = _requests(c)
    if c["op"] == "layout":
        parents = _trees(c, news, random.Random(seed))
        got = {"req": [], "slot": [], "pos": [], "mask": _masks(parents)}
        for b, (m, t) in enumerate(zip(_layout_lens(c, seed), news)):
            got["req"] += [b] * t
            got["slot"] += range(m - t, m)
            got["pos"] += [m - t + x for x in _depths(parents[b])]
        tail = [0] * c["pad"]
        return {k: torch.tensor(x + tail, dtype=torch.int64 if k == "mask" else torch.int32).cuda()
                for k, x in got.items()}
    if c["op"] == "accept":
        n_kept, path, nxt, lens_out = [], [], [], []
        parent, token, target = (s[k].tolist() for k in ("parent", "token", "target"))
        flat = [(s[x], s[x].clone()) for x in ("k", "v")]
        table, first = s["table"].tolist(), 0
        for b, (m, t) in enumerate(zip(lens, news)):
            way = [0]
            while True:
                nxt_row = [i for i in range(way[-1] + 1, t) if parent[first + i] == way[-1]
                           and token[first + i] == target[first + way[-1]]]
                if not nxt_row:
                    break
                way.append(nxt_row[0])
            n_kept.append(len(way))
            path += way + [-1] * (t - len(way))
            nxt.append(target[first + way[-1]])
            lens_out.append(m - t + len(way))
            for to, row in enumerate(way):
                a, z = m - t + row, m - t + to
                for old, now in flat:
                    now[:, table[b][z // c["page"]], z % c["page"]] = old[:, table[b][a // c["page"]], a % c["page"]]
            first += t
        return {"n_kept": _i32(n_kept), "path": _i32(path + [0] * c["pad"]), "next": _i32(nxt),
                "lens_out": _i32(lens_out), "k": flat[0][1], "v": flat[1][1]}
    h, kv, d = c["heads"], c["kv"], c["dim"]
    if c["op"] == "append":
        x = s["qkv"].double().reshape(-1, h + 2 * kv, d)[:s["rows"]]
        q, k, v = x[:, :h].clone(), x[:, h:h + kv].clone(), x[:, h + kv:]
        P, pos = c["rotary"], s["pos"].long()[:s["rows"]]
        for y, w in ((q, "q_norm"), (k, "k_norm")):
            if c["norms"]:
                y /= ((y ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
                y *= s[w].double()
            if P:
                turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
                pairs = y[..., :P].reshape(*y.shape[:2], P // 2, 2) if c["interleaved"] else \
                    y[..., :P].reshape(*y.shape[:2], 2, P // 2).transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
                y[..., :P] = (z if c["interleaved"] else z.transpose(-1, -2)).reshape(*y.shape[:2], P)
        out = {"k": s["k"].double(), "v": s["v"].double(), "q": s["q_out"].double()}
        out["q"][:s["rows"]] = q
        slot, table = s["slot"].tolist(), s["table"].tolist()
        page = torch.tensor([table[b][t // c["page"]] for b, t in zip(s["req"].tolist(), slot) if b >= 0]).cuda()
        place = torch.tensor([t % c["page"] for t in slot if t >= 0]).cuda()
        out["k"][page, place], out["v"][page, place] = k, v
        return out
    out, lse, first = s["out"].double(), s["lse"].double(), 0
    for b, (m, t) in enumerate(zip(lens, news)):
        pages = s["table"][b, :-(-m // c["page"])].long()
        kk, vv = (s[x][pages].flatten(0, 1)[:m].double() for x in ("k", "v"))
        hidden = torch.ones(t, m, dtype=torch.bool)
        hidden[:, :m - t] = False
        for i in range(t if c["tree"] else 0):
            j = i
            while j >= 0:
                hidden[i, m - t + j] = False
                j = s["parents"][b][j]
        if not c["tree"]:
            hidden = torch.arange(m) > torch.arange(m - t, m)[:, None]
        hidden = hidden.cuda()
        for x in range(h):
            score = s["q"][first:first + t, x].double() @ kk[:, x // (h // kv)].T * s["scale"]
            score.masked_fill_(hidden, -math.inf)
            lse[first:first + t, x] = torch.logsumexp(score, -1)
            out[first:first + t, x] = torch.softmax(score, -1) @ vv[:, x // (h // kv)]
        first += t
    return {"out": out, "lse": lse}
