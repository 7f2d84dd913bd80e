"""Attention over the paged cache of keys and values, and its append, against
their definitions in 64 bits, at the sizes, masks, strides and orders where they
can go wrong.

Tolerances.  u = 2^-11 (fp16) or 2^-8 (bf16) is the unit roundoff of the type.
Attention rounds the softmax weights and the output, each by a relative u at
most (rms u / sqrt(3)): the 2-norm of the error is sqrt(2 / 3) u of the
output's, taken as 1.5 u; a single value lies within 12 u of its row's rms plus
its own u.  lse is fp32: a score is a sum of at most 128 products whose sizes
sum to at most |q| |k| scale < 32 here, each of 8 or 16 partial sums rounded or
cut at 2^-22, so 16 x 2^-22 x 32 < 1.3e-4.
The append is exact to fp32 before its one rounding: values within u of
themselves plus 1e-5 of the row's rms (fp16 subnormals: 2^-25)."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F16, BF16 = torch.float16, torch.bfloat16


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


def random_parents(t, g):
    return [-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, t)]


def masks_of(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def signed(m):
    return m - (1 << 64) if m >> 63 else m


def pools(pages, page, kv, D, dtype, order, pad=0):
    """Key and value pools full of NaN as views [pages][page][kv][D]."""
    def one():
        if order == "token":
            return torch.full((pages, page, kv + pad, D), math.nan, dtype=dtype, device="cuda")[:, :, :kv]
        if order == "head":
            return torch.full((pages, kv, page + pad, D), math.nan, dtype=dtype, device="cuda").transpose(1, 2)[:, :page]
        if order == "outer":  # a head's pages together
            return torch.full((kv, pages, page, D), math.nan, dtype=dtype, device="cuda").permute(1, 2, 0, 3)
        raise ValueError(order)
    if order == "joint":  # keys and values of a page side by side
        both = torch.full((pages, 2, page, kv, D), math.nan, dtype=dtype, device="cuda")
        return both[:, 0], both[:, 1]
    return one(), one()


def make(lens, news, heads=8, kv=2, D=128, dtype=F16, page=64, order="token", tree=False, seed=0, pad=0, spare=0):
    """Inputs of one call; cache positions nobody may use hold NaN, table entries
    past a request's pages name nothing, `pad` rows behind the last request."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cg = torch.Generator().manual_seed(seed)
    B = len(lens)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    per = max(1, -(-max(max(lens), 1) // page)) + spare
    pages = B * per + 3
    k, v = pools(pages, page, kv, D, dtype, order, pad=1 if spare else 0)
    table = torch.randperm(pages, generator=g, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    s = dict(lens=lens, news=news, heads=heads, kv=kv, D=D, dtype=dtype, K=[], V=[], pad=pad)
    for b, n in enumerate(lens):
        s["K"].append(normal(n, kv, D))
        s["V"].append(normal(n, kv, D))
        at = torch.arange(n, device="cuda")
        k[table[b, at // page].long(), at % page] = s["K"][b]
        v[table[b, at // page].long(), at % page] = s["V"][b]
    need = i32([-(-n // page) for n in lens])
    table[torch.arange(per, device="cuda")[None] >= need[:, None]] = -7
    N = sum(news) + pad
    s["cache"] = _spx().KvCache(k, v, table, i32(lens))
    s["q_start"] = i32([sum(news[:i]) for i in range(B + 1)])
    s["max_q"], s["max_len"] = max(max(news), 1), max(max(lens), 1)
    s["q"], s["scale"] = normal(N, heads, D, std=1.5), 1 / math.sqrt(D)
    s["parents"] = [random_parents(t, cg) if t else [] for t in news] if tree else None
    s["masks"] = [masks_of(p) for p in s["parents"]] if tree else None
    return s


def mask_tensor(s):
    return torch.tensor([signed(m) for ms in s["masks"] for m in ms] + [-1] * s["pad"], dtype=torch.int64,
                        device="cuda") if s["masks"] is not None else None


def call(s, causal=True, q=None, out=None, ws=None, lse=True, stream=None, max_q=None, max_len=None, wait_budget_ns=0):
    spx = _spx()
    q = s["q"] if q is None else q
    out = torch.full(q.shape, 7.0, dtype=s["dtype"], device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    mq, ml = max_q or s["max_q"], s["max_len"] if max_len is None else max_len
    ws = spx.new_kv_workspace(q, s["cache"], mq, ml, stream) if ws is None else ws
    args, keep = spx.kv_attention_args(q, s["cache"], s["q_start"], mq, ml, s["scale"], out, ws, causal=causal,
                                       tree=mask_tensor(s), lse=lse, wait_budget_ns=wait_budget_ns)
    (stream or torch.cuda.current_stream()).wait_stream(torch.cuda.current_stream())
    spx.spx_kv_attention(args, stream)
    (stream or torch.cuda.current_stream()).synchronize()
    assert spx.spx_workspace_status(ws) == 0
    return out, lse


def seen_by(s, b, causal=True):
    n, t = s["lens"][b], s["news"][b]
    p, i = torch.arange(n), torch.arange(t)[:, None]
    if s["masks"] is not None:
        seen = (p < n - t).expand(t, n).clone()
        for r, m in enumerate(s["masks"][b]):
            for j in range(t):
                if m >> j & 1 and n - t + j >= 0:
                    seen[r, n - t + j] = True
        return seen.cuda()
    return (p < (n - t + i + 1 if causal else n + 0 * i)).cuda()


def reference(s, causal=True):
    outs, lses, first = [], [], 0
    g = s["heads"] // s["kv"]
    for b, t in enumerate(s["news"]):
        q = s["q"][first:first + t].double()
        first += t
        seen = seen_by(s, b, causal)
        o, ls = [], []
        for h in range(s["heads"]):
            k, v = s["K"][b][:, h // g].double(), s["V"][b][:, h // g].double()
            sc = torch.where(seen, q[:, h] @ k.T * s["scale"], -math.inf)
            lse = torch.logsumexp(sc, -1) if s["lens"][b] else torch.full((t,), -math.inf, dtype=torch.float64, device="cuda")
            p = torch.where(seen, torch.exp(sc - torch.where(lse > -math.inf, lse, 0.0)[:, None]), 0.0)
            o.append(p @ v)
            ls.append(lse)
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(ls, 1))
    return torch.cat(outs), torch.cat(lses)


def check(s, out, lse, causal=True):
    n = sum(s["news"])
    want, want_lse = reference(s, causal)
    u, err = U[s["dtype"]], (out[:n].double() - want)
    assert torch.isfinite(out[:n]).all()
    rms = want.square().mean(-1, keepdim=True).sqrt()
    assert err.norm() <= 1.5 * u * want.norm(), (err.norm() / want.norm() / u).item()
    assert (err.abs() <= 12 * u * rms + u * want.abs()).all()
    if lse is not None:
        live = want_lse > -math.inf
        assert torch.equal(live, lse[:n] > -math.inf)
        assert ((lse[:n].double() - want_lse)[live].abs() <= 1.3e-4).all()
        assert (lse[n:] == 7).all()
    assert (out[n:] == 7).all()  # rows that no request owns


ONE = [dict(lens=[1], news=[1]), dict(lens=[2], news=[1]), dict(lens=[15], news=[1]), dict(lens=[16], news=[1]),
       dict(lens=[17], news=[1]), dict(lens=[128], news=[1]), dict(lens=[129], news=[1]), dict(lens=[517], news=[1]),
       dict(lens=[20011], news=[1]), dict(lens=[300, 1, 0, 4097, 64], news=[1, 1, 1, 1, 0]),
       dict(lens=[700] * 3 + [50] * 40, news=[1] * 43)]
MANY = [dict(lens=[5], news=[5]), dict(lens=[33, 200], news=[7, 2]), dict(lens=[4113], news=[17]),
        dict(lens=[1000, 64, 63, 2, 0, 515], news=[64, 64, 63, 2, 0, 1]), dict(lens=[131, 130, 129], news=[16, 33, 4]),
        dict(lens=[250, 9000], news=[31, 64])]
LONG = [dict(lens=[128], news=[128]), dict(lens=[300], news=[300]), dict(lens=[129, 600, 1], news=[129, 257, 1]),
        dict(lens=[1200, 2000, 77], news=[511, 1000, 65])]
SHAPES = [dict(heads=4, kv=4, D=128, dtype=F16), dict(heads=8, kv=2, D=128, dtype=BF16, page=16, order="head"),
          dict(heads=7, kv=1, D=64, dtype=F16, page=48, order="outer"), dict(heads=10, kv=2, D=64, dtype=BF16, order="joint"),
          dict(heads=24, kv=1, D=128, dtype=F16, page=128), dict(heads=64, kv=1, D=128, dtype=BF16, page=32)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sizes", ONE, ids=str)
def test_one_token(sizes, shape):
    s = make(**sizes, **shape, pad=2, spare=1)
    check(s, *call(s))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sizes", MANY, ids=str)
@pytest.mark.parametrize("mode", ["tree", "causal", "full"])
def test_several_tokens(sizes, shape, mode):
    s = make(**sizes, **shape, tree=mode == "tree", pad=3)
    check(s, *call(s, causal=mode != "full"), causal=mode != "full")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sizes", LONG, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(sizes, shape, causal):
    s = make(**sizes, **shape, pad=1)
    check(s, *call(s, causal=causal), causal=causal)


@pytest.mark.parametrize("t", [1, 4, 40, 200])
def test_rows_that_see_nothing(t):
    """More rows than the request has tokens: the first ones see nothing (causal)."""
    s = make([max(t // 2, 0), 3], [t, 2], heads=8, kv=2)
    check(s, *call(s))
    s = make([0, 0], [t, t], heads=8, kv=2)
    out, lse = call(s)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("t,base", [(8, 100), (64, 300), (64, 0), (20, 0)])
def test_masks_with_nothing_and_with_all(t, base):
    """Masks are any 64 bits: rows that see no row of the tree, not even themselves, rows that see all, and bits of
    rows that are not there."""
    s = make([base + t], [t], heads=8, kv=2, tree=True)
    g = torch.Generator().manual_seed(3)
    s["masks"] = [[0 if i % 3 == 0 else (1 << 64) - 1 if i % 3 == 1 else
                   int(torch.randint(0, 1 << 62, (1,), generator=g)) for i in range(t)]]
    out, lse = call(s)
    check(s, out, lse)
    if base == 0:
        assert (out[::3] == 0).all() and (lse[::3] == -math.inf).all()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("t,g", [(6, 1), (6, 4), (64, 4), (200, 4)])
def test_values_that_are_not_finite(t, g, where, value):
    """A token that holds one changes the rows that see it, and no others."""
    bad = t - 4
    for tree in (False, True) if t <= 64 else (False,):
        s = make([300 + t], [t], heads=2 * g, kv=2, tree=tree)
        clean, clean_lse = call(s)
        at = 300 + bad
        page = int(s["cache"].block_table[0, at // 64])
        buf = s["cache"].k if where == "key" else s["cache"].v
        buf[page, at % 64, 1, 5:7] = value
        out, lse = call(s)
        seen = seen_by(s, 0)[:, at]
        assert torch.equal(out[:, :g], clean[:, :g])  # the other key head
        assert torch.equal(out[~seen], clean[~seen]) and torch.equal(lse[~seen], clean_lse[~seen])
        assert seen.any() and not seen.all()
        if where == "value":
            assert not torch.isfinite(out[seen][:, g:, 5:7]).any()
            assert torch.equal(lse, clean_lse)
        else:  # an infinite score is a weight of 0 or a NaN
            touched = (out[seen][:, g:] != clean[seen][:, g:]).any(-1) | ~torch.isfinite(out[seen][:, g:]).all(-1)
            assert touched.all()


def test_an_infinity_of_a_prefix_reaches_every_row():
    s = make([400], [5], heads=8, kv=2)
    s["cache"].v[int(s["cache"].block_table[0, 1]), 3, 0, 9] = math.inf
    out, _ = call(s)
    assert not torch.isfinite(out[:, :4, 9]).any() and torch.isfinite(out[:, 4:]).all()


@pytest.mark.parametrize("t", [1, 20, 150])
def test_large_scores(t):
    """Scores of both signs, beyond fp16's range of exponents: no overflow, and far ones do not matter."""
    s = make([700], [t], heads=8, kv=2, D=64)
    s["q"] = s["q"] * 60
    out, lse = call(s)
    want, want_lse = reference(s)
    assert torch.isfinite(out).all()
    # a score of 400 moves by 2^-22 of its products' sizes: its weight by 1e-3
    assert (lse.double() - want_lse).abs().max() <= 16 * 2.0 ** -22 * 60 * 32
    assert (out.double() - want).abs().max() <= 2e-2


@pytest.mark.parametrize("t", [1, 30, 140])
def test_missing_pages_read_as_zeros(t):
    s = make([600], [t], heads=8, kv=2)
    s["cache"].block_table[0, 2] = 10 ** 6
    for x in ("K", "V"):
        s[x][0][128:192] = 0
    check(s, *call(s))


@pytest.mark.parametrize("t", [1, 17, 64, 300])
def test_strides_of_queries_and_outputs(t):
    s = make([t + 200, 50], [t, 1], heads=8, kv=2)
    N = s["q"].shape[0]
    wide = torch.full((N, 12, 128), math.nan, dtype=F16, device="cuda")
    wide[:, 2:10] = s["q"]
    place = torch.full((N, 11, 128), 7.0, dtype=F16, device="cuda")
    out, lse = call(s, q=wide[:, 2:10], out=place[:, 1:9])
    assert (place[:, 0] == 7).all() and (place[:, 9:] == 7).all()
    check(s, out, lse)
    # lse is not needed
    again, _ = call(s, lse=False)
    assert torch.equal(again, out)


@pytest.mark.parametrize("t", [1, 17, 300])
def test_counts_beyond_the_bounds_are_cut(t):
    """max_q and max_len below what q_start and lens say: no access leaves a buffer."""
    s = make([t + 300], [t], heads=8, kv=2)
    out, _ = call(s, max_len=t + 100)
    assert torch.isfinite(out).all()
    if t > 1:
        out, _ = call(s, max_q=t - 1)
        assert (out[t - 1:] == 7).all() and torch.isfinite(out).all()
    for starts in ([-5, 10 ** 9], [10 ** 9, -5], [3, 1], [-2 ** 31, 2 ** 31 - 1]):
        s["q_start"].copy_(i32(starts))
        call(s)
    s["q_start"].copy_(i32([0, t]))
    for n in (-5, 2 ** 31 - 1, -2 ** 31):
        s["cache"].lens.fill_(n)
        call(s, max_len=t + 300)


@pytest.mark.parametrize("t,tree", [(1, False), (17, True), (64, True), (257, False)])
def test_graph_stream_and_repetition(t, tree):
    """The same bits from a second call, another stream, a larger workspace and two graphs that share it."""
    s = make([5000, t + 1], [t, t], heads=8, kv=2, dtype=BF16, tree=tree)
    want, want_lse = call(s)
    check(s, want, want_lse)
    for _ in range(3):
        assert torch.equal(call(s)[0], want)
    assert torch.equal(call(s, stream=torch.cuda.Stream())[0], want)
    spx = _spx()
    n = spx.spx_kv_workspace_size(8, 8 * t, t, 9000, 8, 2)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")  # past its first part anything may lie in it
    ws[:spx.SPX_KV_WORKSPACE_ZERO] = 0
    assert torch.equal(call(s, ws=ws)[0], want)
    outs, graphs, keeps = [], [], []
    for i in range(2):
        out = torch.zeros_like(s["q"])
        args, keep = spx.kv_attention_args(s["q"], s["cache"], s["q_start"], t, 5000, s["scale"], out, ws, tree=mask_tensor(s))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            spx.spx_kv_attention(args)
            spx.spx_kv_attention(args)
        outs.append(out)
        graphs.append(g)
        keeps.append((args, keep))
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # lengths are read when the graph runs
    s["cache"].lens.copy_(i32([4000, t]))
    s["lens"], s["K"], s["V"] = [4000, t], [x[:n] for x, n in zip(s["K"], (4000, t))], [x[:n] for x, n in zip(s["V"], (4000, t))]
    graphs[0].replay()
    torch.cuda.synchronize()
    check(s, outs[0], None)


@pytest.mark.parametrize("t", [1, 20, 130])
def test_offsets_beyond_32_bits(t):
    """Pages whose elements lie past 2^31."""
    s = make([200], [t], heads=4, kv=1, D=64, dtype=BF16, page=64)
    step = 2 ** 30
    big = torch.empty(4 * step + 64 * 128, dtype=BF16, device="cuda")
    k = big.as_strided((5, 64, 1, 64), (step, 64, 64, 1))
    v = big[64 * 64:].as_strided((5, 64, 1, 64), (step, 64, 64, 1))
    table = i32([[4, 2, 3, 1]])
    for p in range(4):
        rows = min(64, 200 - 64 * p)
        k[table[0, p], :rows] = s["K"][0][64 * p:64 * p + rows]
        v[table[0, p], :rows] = s["V"][0][64 * p:64 * p + rows]
    s["cache"] = _spx().KvCache(k, v, table, i32([200]))
    check(s, *call(s))


@pytest.mark.parametrize("page", [16, 80, 112, 256, 1024])
@pytest.mark.parametrize("t,tree", [(1, False), (20, True), (300, False)])
def test_page_sizes(page, t, tree):
    s = make([t + 1100, t + 3], [t, t], heads=8, kv=2, page=page, tree=tree)
    check(s, *call(s))
    s = make([t + 5], [t], heads=5, kv=1, D=64, dtype=BF16, page=max(page, -(-(t + 5) // 16) * 16), tree=tree)  # one page holds all
    check(s, *call(s))


@pytest.mark.parametrize("t", [1, 6, 40])
def test_long_caches(t):
    s = make([150001, 70000], [t, t], heads=4, kv=1, D=64, dtype=BF16, page=128, tree=t > 1)
    check(s, *call(s))


def test_two_streams_with_a_workspace_each():
    spx = _spx()
    states = [make([3000] * 4, [t] * 4, heads=8, kv=2, dtype=BF16, tree=tree, seed=t) for t, tree in
              ((1, False), (1, False), (64, True), (200, False))]
    want = [call(s)[0] for s in states]
    streams, calls = [torch.cuda.Stream() for _ in states], []
    for s in states:
        out = torch.zeros_like(s["q"])
        ws = spx.new_kv_workspace(s["q"], s["cache"], s["max_q"], s["max_len"])
        calls.append((spx.kv_attention_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                            tree=mask_tensor(s)), out, ws))
    torch.cuda.synchronize()
    for _ in range(50):
        for stream, ((args, keep), out, ws) in zip(streams, calls):
            spx.spx_kv_attention(args, stream)
    torch.cuda.synchronize()
    for ((args, keep), out, ws), w in zip(calls, want):
        assert torch.equal(out, w) and spx.spx_workspace_status(ws) == 0


def test_many_requests():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 400, (1000,), generator=g).tolist()
    s = make(lens, [1 if n else 0 for n in lens], heads=4, kv=2, D=64)
    check(s, *call(s))
    lens = [n + 9 for n in lens[:300]]
    s = make(lens, [1 + n % 9 for n in lens], heads=16, kv=2, D=64, tree=True)
    check(s, *call(s))


# ---------------------------------------------------------------- append --
def rotate(x, cos, sin, interleaved):
    P = 2 * cos.shape[-1]
    a, b = (x[..., 0:P:2], x[..., 1:P:2]) if interleaved else (x[..., :P // 2], x[..., P // 2:P])
    c, s = cos[:, None].double(), sin[:, None].double()
    r = torch.stack([a * c - b * s, b * c + a * s], -1 if interleaved else -2).flatten(-2)
    return torch.cat([r, x[..., P:]], -1)


def near(got, want, dtype):
    rms = want.square().mean(-1, keepdim=True).sqrt()
    return ((got.double() - want).abs() <= U[dtype] * want.abs() + 1e-5 * rms + 2.0 ** -25).all()


@pytest.mark.parametrize("n", [1, 3, 17, 300, 4099])
@pytest.mark.parametrize("dtype,D,P,interleaved,norms,order,page", [
    (F16, 128, 128, False, False, "token", 64), (BF16, 128, 64, True, True, "head", 16), (F16, 64, 64, True, True, "outer", 48),
    (BF16, 64, 16, False, True, "joint", 32), (F16, 128, 0, False, True, "token", 128), (BF16, 64, 0, False, False, "head", 64),
    (BF16, 128, 96, False, True, "token", 64)])
def test_append(n, dtype, D, P, interleaved, norms, order, page):
    spx, g = _spx(), torch.Generator(device="cuda").manual_seed(n)
    (heads, kv), B = (5, 5) if D == 64 else (12, 4), 3
    per = -(-(n + 40) // page)
    k, v = pools(B * per + 1, page, kv, D, dtype, order)
    k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
    v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    table = torch.randperm(B * per + 1, generator=g, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    cache = spx.KvCache(k, v, table, i32([n + 40] * B))
    qkv = torch.randn(n, heads + 2 * kv, D, generator=g, device="cuda").to(dtype)
    req = torch.randint(0, B, (n,), generator=g, device="cuda").to(torch.int32)
    slot = (torch.randperm(n, generator=g, device="cuda") + 7).to(torch.int32)
    pos = torch.randint(0, 1000, (n,), generator=g, device="cuda").to(torch.int32)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)) if norms else (None, None)
    angle = torch.arange(1000, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, max(P, 1), 2, device="cuda") / max(P, 1))
    cos, sin = (angle.cos().float().contiguous(), angle.sin().float().contiguous()) if P else (None, None)
    # rows that are skipped: no slot, a position out of range, no request, a slot past the table
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    stored = live.clone()
    if n > 10:
        slot[2], pos[3], pos[4], req[5], req[6], slot[7] = -1, -3, 1000 if P else -1, -1, B, per * page
        live[2:5] = False
        stored[2:8] = False
        table[1, per // 2] = -1  # a missing page
        stored &= ~((req == 1) & (slot // page == per // 2))
    want_k, want_v = k.double(), v.double()
    x = qkv.double()
    q, kk = x[:, :heads].clone(), x[:, heads:heads + kv].clone()
    for y, w in ((q, wq), (kk, wk)):
        if w is not None:
            y /= (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            y *= w.double()
    if P:
        at = pos.clamp(0, 999).long()
        q, kk = rotate(q, cos[at], sin[at], interleaved), rotate(kk, cos[at], sin[at], interleaved)
    where = (table[req.clamp(0, B - 1).long(), (slot.clamp(0, per * page - 1) // page).long()].long()[stored],
             (slot % page).long()[stored])
    want_k[where], want_v[where] = kk[stored], x[stored][:, heads + kv:]
    changed = torch.zeros(k.shape[:2], dtype=torch.bool, device="cuda")
    changed[where] = True
    before = k.clone()
    q_out = torch.full((n, heads + 1, D), 7.0, dtype=dtype, device="cuda")
    args, keep = spx.kv_append_args(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], req, slot, pos=pos,
                                    q=qkv[:, :heads], q_out=q_out[:, :heads], q_norm=wq, k_norm=wk, cos=cos, sin=sin,
                                    interleaved=interleaved)
    spx.spx_kv_append(args)
    assert near(k, want_k, dtype) and near(q_out[live][:, :heads], q[live], dtype)
    assert torch.equal(v.double(), want_v) and torch.equal(k[~changed], before[~changed])
    assert (q_out[~live] == 7).all() and (q_out[:, heads] == 7).all()
    # in place, and keys alone
    first = q_out[:, :heads].clone()
    kept = qkv[:, :heads].clone()
    k.copy_(before)
    args, keep = spx.kv_append_args(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], req, slot, pos=pos,
                                    q=qkv[:, :heads], q_norm=wq, k_norm=wk, cos=cos, sin=sin, interleaved=interleaved)
    spx.spx_kv_append(args)
    assert torch.equal(qkv[live][:, :heads], first[live]) and torch.equal(qkv[~live][:, :heads], kept[~live])
    stood = k.clone()
    k.copy_(before)
    args, keep = spx.kv_append_args(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], req, slot, pos=pos, k_norm=wk,
                                    cos=cos, sin=sin, interleaved=interleaved)
    spx.spx_kv_append(args)
    assert torch.equal(k, stood)


def test_append_without_positions_turns_by_the_slot():
    spx = _spx()
    k, v = pools(3, 64, 2, 64, F16, "token")
    cache = spx.KvCache(k, v, i32([[2, 0]]), i32([100]))
    x = torch.randn(2, 4, 64, device="cuda").half()
    angle = torch.arange(128, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, device="cuda") / 64)
    cos, sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()
    slot = i32([70, 3])
    args, keep = spx.kv_append_args(cache, x[:, :2], x[:, 2:], i32([0, 0]), slot, cos=cos, sin=sin)
    spx.spx_kv_append(args)
    want = rotate(x[:, :2].double(), cos[slot.long()], sin[slot.long()], False)
    assert near(torch.stack([k[0, 6], k[2, 3]]), want, F16) and torch.equal(torch.stack([v[0, 6], v[2, 3]]), x[:, 2:])
    assert int(torch.isnan(k).all(-1).logical_not().sum()) == 4


def test_binding_refusals():
    spx = _spx()
    s = make([100], [1])
    ws = spx.new_kv_workspace(s["q"], s["cache"], 1, 100)
    out = torch.empty_like(s["q"])
    good = dict(q=s["q"], cache=s["cache"], q_start=s["q_start"], max_q=1, max_len=100, scale=1.0, out=out, ws=ws)
    for bad in (dict(q=s["q"].float()), dict(out=out[:, :4]), dict(q_start=s["q_start"].long()), dict(q=s["q"].cpu()),
                dict(q_start=s["q_start"][:1]), dict(tree=s["q_start"][:1]), dict(lse=torch.empty(1, 3, device="cuda")),
                dict(out=out.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(cache=spx.KvCache(s["cache"].k, s["cache"].v[:1], s["cache"].block_table, s["cache"].lens)),
                dict(cache=spx.KvCache(s["cache"].k, s["cache"].v, s["cache"].block_table[0], s["cache"].lens))):
        with pytest.raises(ValueError):
            spx.kv_attention_args(**{**good, **bad})
    with pytest.raises(spx.SpxError):
        args, keep = spx.kv_attention_args(**{**good, "ws": ws[:100]})
        spx.spx_kv_attention(args)


@pytest.mark.parametrize("fill", [0x7f, 0xff, 0x00, 0x01])
def test_one_workspace_for_calls_of_all_sizes(fill):
    """Whatever an earlier call, or nobody, left behind the workspace's first bytes: requests without rows, with few and
    with many among those of one call, units that cross from block to block and units that do not."""
    spx = _spx()
    states = [make([3000, 40, 0, 2600], [200, 40, 0, 3], heads=8, kv=2, seed=31),
              make([5000, 300, 900], [64, 0, 17], heads=8, kv=2, tree=True, seed=32),
              make([2500, 2500, 130], [1, 65, 129], heads=8, kv=2, dtype=BF16, D=64, seed=33),
              make([260] * 8, [33] * 8, heads=8, kv=8, tree=True, seed=34),
              make([6000, 10], [1, 1], heads=8, kv=2, seed=35),
              make([1500, 1400], [0, 300], heads=4, kv=1, seed=36)]
    size = max(spx.spx_kv_workspace_size(len(s["lens"]), len(s["q"]), s["max_q"], s["max_len"], s["heads"], s["kv"], s["D"])
               for s in states)
    ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
    ws[:spx.SPX_KV_WORKSPACE_ZERO] = 0
    for turn in range(2):
        for s in states if turn == 0 else states[::-1]:
            out, lse = call(s, ws=ws)
            check(s, out, lse)
