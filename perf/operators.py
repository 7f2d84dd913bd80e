"""What surrounds the expert layer in one verification step of a speculating
decoder, as measurable operators:

* ``latent_attention``: attention of a few new tokens (draft: 1, verify: the
  drafted tokens and one more) or of a prompt chunk over a paged cache that
  holds one latent vector and one rotated key part per token;
* ``latent_append``: the new tokens' latent vectors normalised, their key part
  (and the queries' part) rotated, and both written to the cache;
* ``token_logprobs``: from the verify pass's logits, the log probability of
  each drafted token, the entropy and the most likely alternatives.

``own`` selects between the plain form (elementary torch operations in 32
bits) and the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

R, P, NOPE, VALUE = 512, 64, 128, 128  # latent width, rotated width, per-head widths
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the draft step of one request early in its answer: launch latency
        dict(name="decode_short", op="attention", dtype="f16", heads=16, batch=1, tokens=1, context=517, ragged=False,
             page=64, folded=False),
        # the draft step of one request with a long document behind it: cache bandwidth
        dict(name="decode_long", op="attention", dtype="f16", heads=16, batch=1, tokens=1, context=65536, ragged=False,
             page=64, folded=False),
        # the verify pass of one request (16 drafted tokens and one more)
        dict(name="verify_one", op="attention", dtype="f16", heads=16, batch=1, tokens=17, context=4113, ragged=False,
             page=64, folded=False),
        # draft steps of many requests of different lengths
        dict(name="decode_batch", op="attention", dtype="bf16", heads=16, batch=64, tokens=1, context=8192,
             ragged=True, page=64, folded=False),
        # verify passes of several requests, fewer drafted tokens, small pages
        dict(name="verify_batch", op="attention", dtype="f16", heads=16, batch=16, tokens=9, context=8191, ragged=True,
             page=32, folded=False),
        # a wide model whose up-projections are folded into its neighbours' weights
        dict(name="decode_folded", op="attention", dtype="bf16", heads=128, batch=32, tokens=1, context=4096,
             ragged=True, page=64, folded=True),
        # a whole prompt at once
        dict(name="prefill", op="attention", dtype="f16", heads=16, batch=1, tokens=4096, context=4096, ragged=False,
             page=64, folded=False),
        # prompt chunks of several requests behind cached text, odd sizes, the smallest pages
        dict(name="prefill_chunks", op="attention", dtype="bf16", heads=16, batch=4, tokens=1021, context=6007,
             ragged=True, page=16, folded=False),
        # the new tokens of one verify pass go to the cache
        dict(name="append_verify", op="append", dtype="f16", heads=16, batch=1, tokens=17, context=4113, page=64),
        # the tokens of prompt chunks go to the cache
        dict(name="append_prompt", op="append", dtype="bf16", heads=16, batch=4, tokens=2048, context=8192, page=16),
        # acceptance of one verify pass: 17 rows of logits over a whole vocabulary
        dict(name="logprobs_verify", op="logprobs", dtype="f32", rows=17, vocab=102400, top=8, masked=False),
        # scores of many requests' tokens, with the alternatives that an API returns
        dict(name="logprobs_batch", op="logprobs", dtype="bf16", rows=1088, vocab=102400, top=20, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = [work(c) for c in listed()]
    limits = {op: [max(w[k] for w, c in zip(top, listed()) if c["op"] == op) for k in ("bytes", "flops")]
              for op in ("attention", "append", "logprobs")}
    while True:
        op = rng.choice(["attention", "attention", "attention", "append", "logprobs"])
        if op == "attention":
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=rng.choice([8, 16, 16, 16, 20, 32, 128]),
                     batch=_log(rng, 1, 64), tokens=rng.choice([1, rng.randint(2, 33), _log(rng, 34, 4096)]),
                     context=_log(rng, 64, 65536), ragged=rng.random() < 0.6, page=rng.choice([16, 32, 48, 64, 128]),
                     folded=rng.random() < 0.25)
            c["context"] = max(c["context"], c["tokens"])
            if c["batch"] * c["context"] > 1 << 19 or c["batch"] * c["tokens"] * c["context"] * c["heads"] > 1 << 29:
                continue
            if c["folded"] and c["tokens"] > 33:  # folded weights have no expanded form
                continue
        elif op == "append":
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=rng.choice([8, 16, 16, 32]),
                     batch=_log(rng, 1, 16), tokens=_log(rng, 1, 4096), context=_log(rng, 64, 16384),
                     page=rng.choice([16, 32, 48, 64, 128]))
            c["context"] = max(c["context"], c["tokens"])
            if c["batch"] * c["context"] > 1 << 16:
                continue
        else:
            c = dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), rows=_log(rng, 1, 1088),
                     vocab=_log(rng, 1000, 160000), top=rng.choice([1, 2, 5, 8, 20, 32]), masked=rng.random() < 0.3)
        w = work(c)
        if w["bytes"] <= limits[op][0] and w["flops"] <= max(1.0, limits[op][1]):
            return c


def _requests(c):
    """Cached length and new tokens of each request: the same for every seed."""
    B, T, L = c["batch"], c["tokens"], c["context"]
    if not c.get("ragged"):
        return [L] * B, [T] * B
    g = random.Random("%s %s %s %s" % (B, T, L, c["heads"]))
    lens = [L] + [g.randint(max(1, L // 8), L) for _ in range(B - 1)]
    news = [T] + [g.randint(max(1, T // 2), T) for _ in range(B - 1)]
    return lens, [min(t, n) for t, n in zip(news, lens)]


def work(c):
    if c["op"] == "append":
        n, e = c["batch"] * c["tokens"], DTYPES[c["dtype"]].itemsize
        rows = min(c["context"], c["batch"] * c["tokens"])
        return {"bytes": n * (2 * (R + P) * e + 8) + n * c["heads"] * 2 * (NOPE + P) * e + rows * P * 4 + R * e,
                "flops": n * (4.0 * R + 3 * P + 3 * P * c["heads"])}
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * DTYPES[c["dtype"]].itemsize + c["rows"] * (12 + 8 * c["top"]), "flops": 6.0 * n}
    h, e = c["heads"], 2
    lens, news = _requests(c)
    pairs = sum(t * (n - t) + t * (t + 1) // 2 for n, t in zip(lens, news))
    tot, n = sum(lens), sum(news)
    if c["folded"]:
        flops = 2.0 * h * pairs * (2 * R + P)
        size = n * h * (2 * R + P) * e
    else:
        absorbed = 2.0 * h * (pairs * (2 * R + P) + n * R * (NOPE + VALUE))
        expanded = 2.0 * h * (pairs * (NOPE + P + VALUE) + tot * R * (NOPE + VALUE))
        flops = min(absorbed, expanded)
        size = n * h * (NOPE + P + VALUE) * e + h * (NOPE + VALUE) * R * e
    return {"bytes": size + tot * (R + P) * e + 4 * (tot // c["page"] + c["batch"]), "flops": flops}


# ----------------------------------------------------------------- inputs --
def _tables(c, g):
    """A cache with every request's pages at random places."""
    per = -(-c["context"] // c["page"])
    pages = per * c["batch"]
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    return pages, perm.reshape(c["batch"], per).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"] == "logprobs":
        s["logits"] = normal(c["rows"], c["vocab"], std=3.0)
        if c["masked"]:  # a grammar leaves one token in ten, and for the last row none
            keep = torch.rand(c["rows"], c["vocab"], generator=g, device="cuda") < 0.1
            keep[-1] = False
            s["logits"].masked_fill_(~keep, -math.inf)
        s["ids"] = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device="cuda").to(torch.int32)
        s["logp"], s["entropy"] = torch.empty(2, c["rows"], device="cuda").unbind()
        s["top_logp"] = torch.empty(c["rows"], c["top"], device="cuda")
        s["top_ids"] = torch.empty(c["rows"], c["top"], dtype=torch.int32, device="cuda")
        return s
    pages, s["table"] = _tables(c, g)
    s["cache"] = normal(pages, c["page"], R + P)
    h, B = c["heads"], c["batch"]
    if c["op"] == "append":
        n = B * c["tokens"]
        s["kv"] = normal(n, R + P, std=0.7)
        s["q"] = normal(n, h, NOPE + P)
        s["w_norm"] = (1 + 0.1 * torch.randn(R, generator=g, device="cuda")).to(dt)
        angle = torch.arange(c["context"], device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, P, 2, device="cuda", dtype=torch.float64) / P)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["req"] = torch.arange(n, device="cuda", dtype=torch.int32) // c["tokens"]
        s["pos"] = torch.arange(n, device="cuda", dtype=torch.int32) % c["tokens"] + (c["context"] - c["tokens"])
        s["lens"] = torch.full((B,), c["context"], device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty_like(s["q"])
        return s
    lens, news = _requests(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    s["max_q"], s["max_len"], n = max(news), max(lens), sum(news)
    s["scale"] = 1.0 / math.sqrt(NOPE + P)
    if c["folded"]:
        s["q"] = torch.cat([normal(n, h, R, std=0.5), normal(n, h, P)], -1)
    else:
        s["q"] = normal(n, h, NOPE + P)
        s["w_uk"] = normal(h, NOPE, R, std=R ** -0.5)
        s["w_uv"] = normal(h, VALUE, R, std=R ** -0.5)
    s["out"] = torch.empty(n, h, R if c["folded"] else VALUE, dtype=dt, device="cuda")
    return s


# -------------------------------------------------------------------- run --
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "append": _own_append, "logprobs": _own_logprobs}[op](state)
    return {"attention": _plain_attention, "append": _plain_append, "logprobs": _plain_logprobs}[op](state)


def _own_attention(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:  # a program keeps its workspace and its argument block from call to call
        cache = spx.LatentCache(s["cache"], s["table"], s["lens"], R, P)
        ws = spx.new_latent_workspace(s["q"], cache, s["max_q"], s["max_len"], s.get("w_uk"), s.get("w_uv"))
        s["call"] = spx.latent_args(s["q"], cache, s["q_start"], s["max_q"], s["max_len"], s["scale"], s["out"], ws,
                                    w_uk=s.get("w_uk"), w_uv=s.get("w_uv"), causal=True)
    spx.spx_latent_attention(s["call"][0])
    return s["out"]


def _own_append(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:
        cache = spx.LatentCache(s["cache"], s["table"], s["lens"], R, P)
        s["call"] = spx.latent_append_args(cache, s["kv"], s["req"], s["pos"], w_norm=s["w_norm"], eps=EPS,
                                           cos=s["cos"], sin=s["sin"], interleaved=True, q=s["q"], q_out=s["q_out"])
    spx.spx_latent_append(s["call"][0])
    return {"cache": s["cache"], "q": s["q_out"]}


def _own_logprobs(s):
    from quantized_expert_gb300 import spx
    if "call" not in s:
        s["call"] = spx.logprobs_args(s["logits"], s["ids"], s["logp"], s["entropy"], s["top_ids"], s["top_logp"])
    spx.spx_token_logprobs(s["call"][0])
    return {k: s[k] for k in ("logp", "entropy", "top_ids", "top_logp")}


def _plain_attention(s):
    c, lens, q_start = s["case"], s["lens"].long(), s["q_start"].long()
    B, T, L = lens.numel(), s["max_q"], s["max_len"]
    at = torch.arange(L, device="cuda")
    page = s["table"].long()[:, at // c["page"]]                            # [B][L]
    kv = s["cache"][page, at % c["page"]].float()                           # [B][L][R + P]
    i = torch.arange(T, device="cuda")
    news = q_start[1:] - q_start[:-1]
    row = (q_start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B][T]
    q = s["q"].float()[row]                                                 # [B][T][h][.]
    lat, rot = kv[..., :R], kv[..., R:]
    if c["folded"]:
        score = q.permute(0, 2, 1, 3).flatten(1, 2) @ kv.transpose(1, 2)    # [B][h * T][L]
        score = score.reshape(B, c["heads"], T, L)
        value = lat[:, None]
    else:
        key = (lat[:, None] @ s["w_uk"].float().transpose(1, 2))            # [B][h][L][NOPE]
        value = (lat[:, None] @ s["w_uv"].float().transpose(1, 2))          # [B][h][L][VALUE]
        qh = q.permute(0, 2, 1, 3)                                          # [B][h][T][.]
        score = qh[..., :NOPE] @ key.transpose(2, 3) + qh[..., NOPE:] @ rot[:, None].transpose(2, 3)
    score = score * s["scale"]
    seen = at < (lens[:, None] - news[:, None] + i + 1)[..., None]          # [B][T][L]
    score = score.masked_fill(~seen[:, None], -math.inf)
    e = torch.exp(score - score.max(-1, keepdim=True).values.clamp(min=-1e30))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (p.flatten(1, 2) @ value[:, 0]).reshape(B, c["heads"], T, R) if c["folded"] else p @ value
    new = i < news[:, None]
    return out.permute(0, 2, 1, 3)[new].to(s["q"].dtype)


def _plain_append(s):
    c, dt = s["case"], s["kv"].dtype
    kv, pos = s["kv"].float(), s["pos"].long()
    lat = kv[:, :R]
    lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["w_norm"].float()
    cos, sin = s["cos"][pos], s["sin"][pos]

    def rotate(x, cos, sin):
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)

    page = s["table"].long()[s["req"].long(), pos // c["page"]]
    s["cache"][page, pos % c["page"]] = torch.cat([lat, rotate(kv[:, R:], cos, sin)], -1).to(dt)
    q = s["q"].float()
    s["q_out"].copy_(torch.cat([q[..., :NOPE], rotate(q[..., NOPE:], cos[:, None], sin[:, None])], -1))
    return {"cache": s["cache"], "q": s["q_out"]}


def _plain_logprobs(s):
    k, x = s["case"]["top"], s["logits"].float()
    m = x.max(-1, keepdim=True).values
    some = m > -math.inf
    m = torch.where(some, m, torch.zeros_like(m))
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    log_z = torch.where(some, m + torch.log(z.clamp(min=1e-38)), torch.zeros_like(m))
    d = torch.where(e > 0, x - m, torch.zeros_like(x))
    entropy = torch.where(some, torch.log(z.clamp(min=1e-38)) - (e * d).sum(-1, keepdim=True) / z.clamp(min=1e-38),
                          torch.zeros_like(m))
    logp = x.gather(-1, s["ids"].long()[:, None]) - log_z
    top, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    return {"logp": logp[:, 0], "entropy": entropy[:, 0], "top_ids": ids[:, :k].to(torch.int32).contiguous(),
            "top_logp": (top[:, :k] - log_z).contiguous()}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    """The operators' definitions in 64 bits, request by request."""
    s, c = prepare(case, seed), case
    if c["op"] == "logprobs":
        logp, ent, top = [], [], []
        for x, t in zip(s["logits"], s["ids"].tolist()):
            x = x.double()
            if not bool((x > -math.inf).any()):
                logp.append(x[t])
                ent.append(x.new_zeros(()))
                top.append(x[:c["top"]])
                continue
            z = torch.logsumexp(x, 0)
            logp.append(x[t] - z)
            live = x[x > -math.inf] - z
            ent.append(-(live.exp() * live).sum())
            top.append(torch.topk(x, c["top"]).values - z)
        return {"logp": torch.stack(logp), "entropy": torch.stack(ent), "top_ids": None, "top_logp": torch.stack(top)}
    if c["op"] == "append":
        cache = s["cache"].double()
        x = s["kv"].double()
        norm = (x[:, :R] ** 2).sum(-1) / R + EPS
        x[:, :R] = x[:, :R] / norm.sqrt()[:, None] * s["w_norm"].double()
        q = s["q"].double()
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()]
        z = torch.view_as_complex(x[:, R:].reshape(-1, P // 2, 2).contiguous()) * turn
        x[:, R:] = torch.view_as_real(z).reshape(-1, P)
        z = torch.view_as_complex(q[..., NOPE:].reshape(*q.shape[:2], P // 2, 2).contiguous()) * turn[:, None]
        q[..., NOPE:] = torch.view_as_real(z).reshape(*q.shape[:2], P)
        slot = s["table"].long()[s["req"].long(), torch.div(s["pos"].long(), c["page"], rounding_mode="floor")]
        cache.view(-1, R + P)[slot * c["page"] + s["pos"].long() % c["page"]] = x
        return {"cache": cache, "q": q}
    lens, news = _requests(c)
    outs, first = [], 0
    for b, (n, t) in enumerate(zip(lens, news)):
        kv = s["cache"][s["table"][b].long()].flatten(0, 1)[:n].double()
        q = s["q"][first:first + t].double()
        first += t
        if not c["folded"]:
            q = torch.cat([torch.einsum("thd,hdr->thr", q[..., :NOPE], s["w_uk"].double()), q[..., NOPE:]], -1)
        hidden = torch.arange(n, device="cuda") > torch.arange(n - t, n, device="cuda")[:, None]
        lat = []
        for h in range(c["heads"]):
            score = (q[:, h] @ kv.T) * s["scale"]
            lat.append(torch.softmax(score.masked_fill_(hidden, -math.inf), -1) @ kv[:, :R])
        lat = torch.stack(lat, 1)
        outs.append(lat if c["folded"] else torch.einsum("thr,hvr->thv", lat, s["w_uv"].double()))
    return torch.cat(outs)
