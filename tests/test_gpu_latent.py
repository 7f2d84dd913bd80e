"""Latent attention and the latent cache's append against their definitions in
64 bits, at the sizes, masks, strides and orders where they can go wrong.

Tolerances.  u = 2^-11 (fp16) or 2^-8 (bf16) is the unit roundoff of the type.
Independent roundings of relative size at most u (rms u / sqrt(3)) enter at the
output, the softmax weights, the latent queries (absorbed) or the keys and
values (expanded); with scores of variance about 1 each moves the output by at
most that share of its own size.  At most five of them: 2-norm 5 u / sqrt(3) <
3 u, taken as 4 u; a single value lies within six standard deviations of that,
12 u of its row's rms, plus its own rounding.  lse moves by the error of a
score, 6 u / sqrt(3) times the largest score, and the fp32 sums (1e-5)."""
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


def make(lens, news, heads=16, dtype=F16, page=64, R=512, dn=128, dv=128, folded=False, seed=0, max_pages=None,
         token_pad=0, page_pad=0):
    """Inputs of one call; cache positions nobody may use hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, P = len(lens), 64

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    per = max_pages or max(1, -(-max(max(lens), 1) // page))
    pages = B * per + 3
    big = torch.full((pages, (page + page_pad) * (R + P + token_pad)), math.nan, dtype=dtype, device="cuda")
    buf = big.as_strided((pages, page, R + P), (big.stride(0), R + P + token_pad, 1))
    table = torch.randperm(pages, generator=g, device="cuda")[:B * per].to(torch.int32).reshape(B, per).contiguous()
    kv = []
    for b, n in enumerate(lens):
        x = normal(n, R + P)
        kv.append(x)
        at = torch.arange(n, device="cuda")
        buf[table[b, at // page].long(), at % page] = x
    # entries past the request's pages name nothing
    need = torch.tensor([-(-n // page) for n in lens], device="cuda")
    table[torch.arange(per, device="cuda")[None] >= need[:, None]] = -7
    N = sum(news)
    s = dict(lens=lens, news=news, heads=heads, R=R, P=P, dn=dn, dv=dv, folded=folded, dtype=dtype, kv=kv,
             cache=_spx().LatentCache(buf, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), R, P),
             q_start=torch.tensor([sum(news[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda"),
             max_q=max(max(news), 1), max_len=max(max(lens), 1))
    if folded:
        s["q"] = torch.cat([normal(N, heads, R, std=math.sqrt(dn / R)), normal(N, heads, P)], -1)
        s["w_uk"] = s["w_uv"] = None
    else:
        s["q"] = normal(N, heads, dn + P)
        s["w_uk"], s["w_uv"] = normal(heads, dn, R, std=R ** -0.5), normal(heads, dv, R, std=R ** -0.5)
    s["scale"] = 1.0 / math.sqrt(dn + P)
    return s


def call(s, form=0, causal=True, out=None, q=None, ws=None, lse=True, stream=None, wait_budget_ns=0):
    spx = _spx()
    N, width = s["q"].shape[0], s["R"] if s["folded"] else s["dv"]
    out = torch.full((N, s["heads"], width), 7.0, dtype=s["dtype"], device="cuda") if out is None else out
    lse = torch.full((N, s["heads"]), 7.0, device="cuda") if lse else None
    q = s["q"] if q is None else q
    ws = spx.new_latent_workspace(q, s["cache"], s["max_q"], s["max_len"], s["w_uk"], s["w_uv"], form,
                                  stream) if ws is None else ws
    args, keep = spx.latent_args(q, s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                 w_uk=s["w_uk"], w_uv=s["w_uv"], causal=causal, lse=lse, form=form,
                                 wait_budget_ns=wait_budget_ns)
    spx.spx_latent_attention(args, stream)
    (stream or torch.cuda.current_stream()).synchronize()
    assert spx.spx_workspace_status(ws) == 0
    return out, lse


def reference(s, causal=True):
    outs, lses, first = [], [], 0
    R = s["R"]
    for kv, n, t in zip(s["kv"], s["lens"], s["news"]):
        q = s["q"][first:first + t].double()
        first += t
        c, rot = kv[:, :R].double(), kv[:, R:].double()
        i = torch.arange(t, device="cuda")[:, None]
        seen = torch.arange(n, device="cuda")[None] < (n - t + i + 1 if causal else n + 0 * i)
        for h in range(s["heads"]):
            if s["folded"]:
                key, val, qh = torch.cat([c, rot], -1), c, q[:, h]
            else:
                key = torch.cat([c @ s["w_uk"][h].double().T, rot], -1)
                val, qh = c @ s["w_uv"][h].double().T, q[:, h]
            sc = torch.where(seen, (qh @ key.T) * s["scale"], -math.inf)
            lse = torch.logsumexp(sc, -1) if n else torch.full((t,), -math.inf, dtype=torch.float64, device="cuda")
            p = torch.where(seen, torch.exp(sc - torch.where(lse > -math.inf, lse, 0.0)[:, None]), 0.0)
            outs.append((p[:, :, None] * torch.where(seen[:, :, None], val[None], 0.0)).sum(1)
                        if n * t <= 4096 else p @ val)
            lses.append(lse)
    t0 = []
    k = 0
    for t in s["news"]:
        t0.append((torch.stack(outs[k:k + s["heads"]], 1), torch.stack(lses[k:k + s["heads"]], 1)))
        k += s["heads"]
    return torch.cat([a for a, _ in t0]), torch.cat([b for _, b in t0])


def check(s, got, want):
    (out, lse), (ref, rl) = got, want
    u, o = U[s["dtype"]], out.double()
    assert torch.equal(torch.isnan(o), torch.isnan(ref))
    live = ~torch.isnan(ref)
    o, ref = torch.where(live, o, 0.0), torch.where(live, ref, 0.0)
    assert (o - ref).norm() <= 4 * u * ref.norm() + 1e-30, float((o - ref).norm() / ref.norm() / u)
    rms = ref.square().mean(-1, keepdim=True).sqrt()
    over = ((o - ref).abs() - 12 * u * rms - u * ref.abs()).max() if o.numel() else 0
    assert over <= 0, float(over)
    if lse is not None:
        assert torch.equal(torch.isinf(lse), torch.isinf(rl))
        fin = torch.isfinite(rl)
        assert ((lse.double() - rl).abs()[fin] <= 6 / math.sqrt(3) * u * 8 + 1e-5).all()


CASES = [
    # lens, news, heads, page
    ([1], [1], 16, 64),                                    # one token that sees itself
    ([64], [1], 16, 64), ([65], [1], 16, 64), ([63], [1], 1, 16),   # around a tile's and a page's end
    ([517], [1], 16, 64), ([517], [17], 16, 48),
    ([4113], [17], 16, 64), ([3001], [9], 20, 32),         # rows that do not fill their groups
    ([700], [33], 7, 128), ([129], [129], 16, 64),         # a whole short prompt
    ([1000, 1, 64, 333], [1, 1, 1, 1], 16, 64),            # ragged draft steps
    ([900, 0, 17, 2, 130], [5, 0, 17, 2, 3], 16, 16),      # an empty request, all-new requests
    ([0, 40], [3, 2], 16, 16),                             # rows that see nothing at all
    ([2, 50], [5, 9], 16, 16),                             # more new tokens than cached ones
    ([257] * 40, [2] * 40, 4, 64),                         # many short requests
    ([300], [1], 128, 64), ([200, 77], [3, 2], 64, 64),
]


@pytest.mark.parametrize("lens,news,heads,page", CASES)
@pytest.mark.parametrize("dtype,folded", [(F16, False), (BF16, False), (F16, True)])
def test_attention_matches_definition(lens, news, heads, page, dtype, folded):
    s = make(lens, news, heads, dtype, page, folded=folded, seed=len(lens) + heads)
    check(s, call(s), reference(s))


@pytest.mark.parametrize("R", [128, 256, 384])
@pytest.mark.parametrize("dn,dv,folded", [(128, 64, False), (64, 128, False), (64, 64, True)])
def test_widths(R, dn, dv, folded):
    s = make([300, 41], [3, 1], 16, BF16, 32, R=R, dn=dn, dv=dv, folded=folded)
    check(s, call(s), reference(s))


@pytest.mark.parametrize("form", [1, 2])
def test_large_prompt_scores(form):
    s = make([900], [300], 4, F16, 64)
    s["q"] *= 40
    out, lse = call(s, form=form)
    ref, rl = reference(s)
    # scores of deviation 40 carry 40 times the error: 4 u grows to 160 u
    assert (out.double() - ref).norm() <= 160 * U[F16] * ref.norm()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("lens,news", [([517, 65], [17, 1]), ([0, 3], [2, 5])])
def test_not_causal(lens, news):
    s = make(lens, news, 16, F16, 64)
    check(s, call(s, causal=False), reference(s, causal=False))


@pytest.mark.parametrize("lens,news,heads,page", [c for c in CASES if c[2] <= 64])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_expanded_form_matches_definition(lens, news, heads, page, dtype):
    s = make(lens, news, heads, dtype, page, seed=len(lens) + heads)
    check(s, call(s, form=2), reference(s))


@pytest.mark.parametrize("lens,news,heads,page,R", [
    ([256], [256], 4, 64, 512), ([257], [257], 3, 48, 512), ([1000], [700], 5, 16, 512), ([900, 333], [300, 333], 4, 32, 256),
    ([512, 0, 130], [384, 0, 129], 6, 128, 128), ([40], [300], 4, 64, 512), ([1500, 700], [1, 513], 4, 64, 384),
    ([4096], [4096], 2, 64, 512)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(lens, news, heads, page, R, causal):
    """Prompts take the expanded form by themselves; tiles of 128 rows and keys
    that end early, rows that see nothing, requests of other lengths."""
    s = make(lens, news, heads, BF16 if heads % 2 else F16, page, R=R, seed=sum(lens))
    auto = call(s, causal=causal)
    check(s, auto, reference(s, causal))
    assert torch.equal(call(s, form=2, causal=causal)[0], auto[0])


def test_forms_agree_on_masked_values():
    """What a later token holds does not reach the rows before it."""
    for bad in (math.nan, math.inf):
        s = make([700], [300], 4, F16, 64)
        clean, _ = call(s, form=2)
        s["cache"].buf[s["cache"].block_table[0, 650 // 64].long(), 650 % 64] = bad
        out, _ = call(s, form=2)
        assert torch.equal(out[:250], clean[:250])
        if math.isnan(bad):
            assert torch.isnan(out[250:]).all()


def test_long_context_and_batch():
    s = make([20011, 9000, 31, 14000], [1, 2, 17, 4], 16, BF16, 64)
    check(s, call(s), reference(s))


def test_large_scores():
    """Scores of some hundreds: the running maximum carries the sums, weights
    before a new maximum lose all theirs."""
    s = make([1500], [5], 16, F16, 64)
    s["q"] *= 40
    out, lse = call(s, form=1)
    ref, rl = reference(s)
    # scores of deviation 40 carry 40 times the error: 4 u grows to 160 u
    assert (out.double() - ref).norm() <= 160 * U[F16] * ref.norm()
    assert ((lse.double() - rl).abs() <= 160 * U[F16] + 1e-5 * rl.abs()).all()
    assert torch.isfinite(out).all()


def test_rising_and_equal_scores():
    """Scores that rise along the cache (every tile has a new maximum) and
    scores that are all equal (a mean)."""
    s = make([1200], [1], 16, F16, 64, folded=True)
    s["q"].zero_()
    out, lse = call(s)
    check(s, (out, lse), reference(s))
    s["q"][:, :, 0] = 1.0
    ramp = (torch.arange(1200, device="cuda") * 0.25).to(F16)
    s["kv"][0][:, 0] = ramp
    at = torch.arange(1200, device="cuda")
    s["cache"].buf[s["cache"].block_table[0, at // 64].long(), at % 64] = s["kv"][0]
    out, lse = call(s)
    check(s, (out, None), reference(s))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_in_masked_places_stay_there(bad):
    """A drafted token whose latent vector is not finite reaches only the rows
    that see it."""
    s = make([200], [9], 16, F16, 64)
    clean, _ = call(s)
    s["cache"].buf[s["cache"].block_table[0, 195 // 64].long(), 195 % 64] = bad
    out, _ = call(s)
    assert torch.equal(out[:4], clean[:4])
    if math.isnan(bad):
        assert torch.isnan(out[4:]).all()


def test_strides_streams_and_offsets():
    """Padded tokens and pages, queries and results inside wider rows, a stream
    of the caller's, a workspace larger than needed."""
    spx = _spx()
    s = make([517, 130], [3, 2], 16, F16, 48, token_pad=24, page_pad=2)
    N, h = s["q"].shape[:2]
    wide = torch.full((N, h * 192 + 64), math.nan, dtype=F16, device="cuda")
    q = wide[:, 32:32 + h * 192].view(N, h, 192)
    q.copy_(s["q"])
    hold = torch.full((N, h * 128 + 8), 5.0, dtype=F16, device="cuda")
    out = hold[:, 8:].view(N, h, 128)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(spx.spx_latent_workspace_size(4, 100, 17, 4000, h, dn=128, dv=128), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    call(s, out=out, q=q, ws=ws, stream=stream)
    torch.cuda.synchronize()
    check(s, (out, None), reference(s))
    assert (hold[:, :8] == 5).all()


def test_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^32 in the cache."""
    s = make([150], [2], 16, F16, 64)
    big = torch.empty(20 * (1 << 28), dtype=F16, device="cuda")  # 10.7 GB
    buf = big.as_strided((20, 64, 576), (1 << 28, 576, 1))
    table = torch.tensor([[19, 3, 17]], dtype=torch.int32, device="cuda")
    at = torch.arange(150, device="cuda")
    for pg in (3, 17, 19):
        buf[pg] = math.nan
    buf[table[0, at // 64].long(), at % 64] = s["kv"][0]
    s["cache"] = _spx().LatentCache(buf, table, s["cache"].lens, 512, 64)
    check(s, call(s), reference(s))


def test_same_bits_again_and_in_a_graph():
    spx = _spx()
    s = make([3000, 700], [9, 9], 16, F16, 64)
    a, _ = call(s)
    b, _ = call(s)
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    ws = spx.new_latent_workspace(s["q"], s["cache"], s["max_q"], s["max_len"], s["w_uk"], s["w_uv"])
    args, keep = spx.latent_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                 w_uk=s["w_uk"], w_uv=s["w_uv"])
    spx.spx_latent_attention(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spx.spx_latent_attention(args)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)
    # lengths are device data: the captured call follows them
    s["cache"].lens[0] = 1000
    graph.replay()
    torch.cuda.synchronize()
    s["lens"] = [1000, 700]
    s["kv"][0] = s["kv"][0][:1000]
    check(s, (out, None), reference(s))


def test_device_contents_out_of_range_are_cut():
    """Lengths beyond max_len and the table, row bounds beyond N: cut, and the
    in-range part of the call is right."""
    s = make([100, 64], [2, 1], 16, F16, 64)
    want, _ = call(s)
    s["cache"].lens[1] = 1 << 30          # max_len is 100, the table holds 2 pages: row 2 is undefined
    s["q_start"][2] = 1 << 30
    out, _ = call(s)
    assert torch.equal(out[:2], want[:2])


def test_no_rows():
    spx = _spx()
    s = make([30], [1], 16, F16, 64)
    s["q"] = s["q"][:0]
    s["q_start"].zero_()
    out, _ = call(s)
    assert out.shape[0] == 0


# ------------------------------------------------------------------ append --
def append_reference(cache, kv, req, pos, w_norm, eps, cos, sin, inter, q):
    R, P = cache.R, cache.P
    buf = cache.buf.double()

    def turn(x, p):
        if cos is None:
            return x
        c, s = cos[p].double(), sin[p].double()
        a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :P // 2], x[..., P // 2:])
        y, z = a * c - b * s, b * c + a * s
        return torch.stack([y, z], -1).flatten(-2) if inter else torch.cat([y, z], -1)

    qo = q.double() if q is not None else None
    for n, (b, p) in enumerate(zip(req.tolist(), pos.tolist())):
        if p < 0 or (cos is not None and p >= cos.shape[0]):
            continue
        if qo is not None:
            qo[n, :, -P:] = turn(qo[n, :, -P:], p)
        if not 0 <= b < cache.lens.numel() or p // cache.buf.shape[1] >= cache.block_table.shape[1]:
            continue
        pg = int(cache.block_table[b, p // cache.buf.shape[1]])
        if not 0 <= pg < cache.buf.shape[0]:
            continue
        x = kv[n].double()
        c = x[:R]
        if w_norm is not None:
            c = c / (c.square().mean() + eps).sqrt() * w_norm.double()
        buf[pg, p % cache.buf.shape[1]] = torch.cat([c, turn(x[R:], p)])
    return buf, qo


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("R,page,norm,rot,inter,heads,width,inplace", [
    (512, 64, True, True, True, 16, 192, False), (512, 16, True, True, False, 16, 192, True),
    (256, 48, False, True, True, 3, 64, True), (384, 32, True, False, True, 5, 288, False),
    (128, 64, True, True, False, 2, 288, True), (512, 64, True, True, True, 0, 0, False)])
def test_append_matches_definition(dtype, R, page, norm, rot, inter, heads, width, inplace):
    """One rounding per value; fp32 sums of at most 512 squares and one
    reciprocal root add less than 1e-6."""
    spx = _spx()
    g = torch.Generator(device="cuda").manual_seed(R + page)
    N, P, B = 37, 64, 3

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    buf = torch.full((12, page, R + P + 8), 3.0, dtype=dtype, device="cuda")[:, :, :R + P]
    table = torch.randperm(12, generator=g, device="cuda")[:9].to(torch.int32).reshape(3, 3).contiguous()
    table[2, 2] = 99   # names no page: rows there are skipped
    cache = spx.LatentCache(buf, table, torch.zeros(B, dtype=torch.int32, device="cuda"), R, P)
    kv = normal(N, R + P + 16)[:, :R + P]
    kv[5, :R] = 0      # a latent vector of zeros: eps keeps the norm finite
    slots = torch.randperm(3 * page * B, generator=g, device="cuda")[:N]
    req, pos = (slots // (3 * page)).to(torch.int32), (slots % (3 * page)).to(torch.int32)
    pos[3], req[7], pos[11] = -1, 3, 3 * page
    req[13] = -1
    angle = torch.rand(3 * page, P // 2, generator=g, device="cuda") * 6
    cos, sin = (angle.cos().contiguous(), angle.sin().contiguous()) if rot else (None, None)
    w = normal(R) if norm else None
    q = normal(N, heads, width) if heads else None
    q_out = None if q is None else q.clone() if inplace else torch.zeros_like(q)
    want, wq = append_reference(cache, kv, req, pos, w, 1e-6, cos, sin, inter, q)
    args, keep = spx.latent_append_args(cache, kv, req, pos, w_norm=w, eps=1e-6, cos=cos, sin=sin, interleaved=inter,
                                        q=q_out if inplace else q, q_out=q_out)
    spx.spx_latent_append(args)
    torch.cuda.synchronize()
    u = U[dtype]
    # a rotated value is a difference of two products: its error is relative to their size
    assert ((cache.buf.double() - want).abs() <= u * want.abs() + 1e-6 * 10).all()
    if q is not None:
        done = (pos >= 0) & ((pos < 3 * page) if rot else (pos > -9))
        assert ((q_out.double() - wq).abs()[done] <= u * wq.abs()[done] + 1e-6 * 10).all()
        skipped = q_out[~done]
        assert torch.equal(skipped, q[~done] if inplace else torch.zeros_like(skipped))
    full = buf.as_strided((12, page, R + P + 8), (page * (R + P + 8), R + P + 8, 1))
    assert (full[:, :, R + P:] == 3).all()


def test_append_then_attend():
    """A verify step: append the new tokens, attend, take rejected ones back by
    a smaller length, append others."""
    spx = _spx()
    s = make([300], [4], 16, F16, 64, max_pages=8)
    cache = s["cache"]
    cache.block_table[0, 5:] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    free = [i for i in range(cache.buf.shape[0]) if i not in cache.block_table[0, :5].tolist()]
    cache.block_table[0, 5:] = torch.tensor((free * 3)[:3], dtype=torch.int32, device="cuda")
    kv = torch.randn(4, 576, device="cuda").to(F16)
    pos = torch.arange(298, 302, dtype=torch.int32, device="cuda")  # the last two replace rejected tokens
    args, keep = spx.latent_append_args(cache, kv, torch.zeros(4, dtype=torch.int32, device="cuda"), pos)
    spx.spx_latent_append(args)
    cache.lens.fill_(302)
    s["kv"][0] = torch.cat([s["kv"][0][:298], kv])
    s["lens"], s["max_len"] = [302], 302
    check(s, call(s), reference(s))
