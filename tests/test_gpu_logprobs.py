"""Log probabilities of given tokens, entropy and alternatives against their
definitions in 64 bits.

Tolerance: fp32 sums of n terms of one sign, in pairs of partial sums, err by
less than 64 * 2^-24 relative whatever n <= 2^20 (partial sums of a thread, a
warp, a block), exponentials by 2 ulp times the size of their argument (at most
100 * 2^-24); a difference x - log_z by 2^-24 of its larger operand.  Together
below 2e-5 of max(1, |x|, |log_z|)."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
TOL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from quantized_expert_gb300 import build, spx
    build.build()
    spx.load()
    yield


def call(x, ids, k, stream=None):
    from quantized_expert_gb300 import spx
    N = x.shape[0]
    logp, ent = torch.full((N,), 9.0, device="cuda"), torch.full((N,), 9.0, device="cuda")
    ti = torch.full((N, k), -5, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((N, k), 9.0, device="cuda") if k else None
    args, keep = spx.logprobs_args(x, ids, logp if ids is not None else None, ent, ti, tl)
    spx.spx_token_logprobs(args, stream)
    torch.cuda.synchronize()
    return logp, ent, ti, tl


def same(got, want, scale):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (got, want)
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
    ok = torch.isfinite(want)
    scale = scale.expand_as(want)[ok]
    assert ((got - want).abs()[ok] <= TOL * scale).all(), float(((got - want).abs()[ok] / scale).max())


def check(x, ids, k, got):
    logp, ent, ti, tl = got
    d = x.double()
    none = (d == -math.inf).all(-1)
    lz = torch.logsumexp(d, -1)
    lz0 = torch.where(none, 0.0, lz)
    size = torch.maximum(torch.where(torch.isfinite(d), d.abs(), 0.0).amax(-1), torch.ones(1, device="cuda").double())
    p = torch.exp(d - lz0[:, None])
    t = torch.where(p > 0, d - lz0[:, None], 0.0)
    want_e = torch.where(none, 0.0, -(p * t).sum(-1))
    want_e = torch.where(torch.isnan(lz) | (lz == math.inf), math.nan, want_e)
    same(ent, want_e, size)
    if ids is not None:
        ok = (ids >= 0) & (ids < x.shape[1])
        v = d.gather(1, ids.long().clamp(0, x.shape[1] - 1)[:, None])[:, 0] - lz0
        same(logp, torch.where(ok, v, math.nan), size)
    if k:
        order = torch.sort(x.float().nan_to_num(nan=math.inf, posinf=3.4e38, neginf=-math.inf), dim=-1,
                           descending=True, stable=True).indices[:, :k]
        assert torch.equal(ti.long(), order)
        same(tl, d.gather(1, order) - lz0[:, None], size[:, None])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (1, 5, 5), (3, 31, 2), (2, 33, 32), (17, 1000, 8), (5, 32003, 20),
                                   (1, 102400, 8), (17, 102400, 0), (300, 4097, 1), (2, 260001, 32)])
def test_matches_definition(dtype, N, V, k):
    g = torch.Generator(device="cuda").manual_seed(V + k)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    check(x, ids, k, call(x, ids, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 3001, 70000])
def test_ties_masks_and_extremes(dtype, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    big = torch.finfo(dtype).max
    x = (torch.randn(12, V, generator=g, device="cuda") * 3).to(dtype)
    x[0] = 1.5                                # all equal: the first k
    x[1] = -math.inf                          # nothing left
    x[2] = -math.inf
    x[2, V - 1] = 0.25                        # one left, fewer than k
    x[3] = -big                               # the type's lowest value everywhere
    x[4, ::2] = -big
    x[5] = (torch.arange(V, device="cuda") % 2).to(dtype)      # two values
    x[6] = 0.0
    x[6, ::3] = -0.0                          # signed zeros tie
    x[7] = (-torch.arange(V, device="cuda") / 64).to(dtype)    # falling: the first ones
    x[8] = (torch.arange(V, device="cuda") / 64).to(dtype)     # rising: the last ones
    x[9] = 0
    x[9, V // 2] = 60000.0                    # a certain token
    x[10, V // 3] = math.nan
    x[10, V // 2] = math.nan
    x[11, : V // 2] = -math.inf               # half masked
    ids = torch.randint(0, V, (12,), generator=g, device="cuda").to(torch.int32)
    ids[0], ids[4], ids[5], ids[9] = -1, V, V - 1, V // 2
    k = 20
    check(x, ids, k, call(x, ids, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [77, 5003, 66000])
def test_lowest_and_infinite_masks_together(dtype, V):
    """Whole stretches at the type's lowest value, next to -inf and to ordinary logits; rows of
    nothing but those two; values between them; few that are left."""
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    big = torch.finfo(dtype).max
    x = (torch.randn(10, V, generator=g, device="cuda") * 3).to(dtype)
    x[0, 5: V - 3] = -big
    x[1, : V // 2] = -big
    x[1, V // 2: V - 2] = -math.inf
    x[2] = -math.inf
    x[2, ::3] = -big                            # uniform over a third
    x[3] = -math.inf
    x[3, V - 1] = -big                          # one left, at the lowest value
    x[4] = -big
    x[4, V // 3] = -big / 2
    x[5] = -big / 2                             # all equal and low
    x[6] = -math.inf
    x[6, V // 2: V // 2 + 3] = 1.0
    x[7, 1::2] = -big / 3
    x[8, 4:] = -math.inf
    x[8, :4] = big / 2                          # large ones
    x[9, : V - 1] = -big
    x[9, V - 1] = -100.0
    ids = torch.randint(0, V, (10,), generator=g, device="cuda").to(torch.int32)
    ids[3], ids[6] = V - 1, V // 2
    k = 8
    check(x, ids, k, call(x, ids, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e5, 9e5, 3e6, 1e8, 1e20, 1e37])
def test_large_logits(dtype, size):
    g = torch.Generator(device="cuda").manual_seed(11)
    x = (torch.randn(4, 9000, generator=g, device="cuda") * 0.25 * size).to(dtype)
    x[1] = x[1].abs()
    x[2] = -x[2].abs() - size
    x[3, ::7] = size
    ids = torch.randint(0, 9000, (4,), generator=g, device="cuda").to(torch.int32)
    check(x, ids, 5, call(x, ids, 5))


def test_infinite_logit():
    x = torch.zeros(1, 100, device="cuda")
    x[0, 7] = math.inf
    logp, ent, ti, tl = call(x, torch.tensor([3], dtype=torch.int32, device="cuda"), 2)
    assert logp[0] == -math.inf and torch.isnan(ent[0]) and ti[0].tolist() == [7, 0]
    assert torch.isnan(tl[0, 0]) and tl[0, 1] == -math.inf


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 3), (3, 5), (7, 1)])
def test_strides_and_alignment(dtype, shift, pad):
    g = torch.Generator(device="cuda").manual_seed(shift)
    hold = (torch.randn(9, 5003 + shift + pad, generator=g, device="cuda") * 2).to(dtype)
    x = hold[:, shift:shift + 5003]
    ids = torch.arange(9, dtype=torch.int32, device="cuda") * 500
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    check(x, ids, 8, call(x, ids, 8, stream))


def test_optional_outputs_and_repetition():
    from quantized_expert_gb300 import spx
    x = torch.randn(4, 3000, device="cuda")
    only = torch.zeros(4, device="cuda")
    args, keep = spx.logprobs_args(x, entropy=only)
    spx.spx_token_logprobs(args)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, b = call(x, ids, 5), call(x, ids, 5)
    assert torch.equal(only, a[1])
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_past_32_bits():
    """Rows that start beyond 2^32 elements."""
    hold = torch.empty(5 * (1 << 30), dtype=torch.float16, device="cuda")  # 10.7 GB
    x = hold.as_strided((5, 1000), (1 << 30, 1))
    x.copy_(torch.randn(5, 1000, device="cuda"))
    ids = torch.arange(5, dtype=torch.int32, device="cuda")
    check(x, ids, 3, call(x, ids, 3))
