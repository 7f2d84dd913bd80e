"""Log probabilities and entropy of rows whose logits share a large offset, or
hold masks of the type's lowest value: neither depends on the offset or on what
is masked, and no tolerance here grows with them.

Tolerance.  The weights' sum and the sum weighted by the exponents carry a
relative error of at most e = 1e-5 (fp32 sums of n <= 2^20 terms in partial sums
64 * 2^-24; exponentials and the rounding of their arguments 100 * 2^-24).  A log
probability is a difference of an exact distance from the reference (rounded
once) and ln z: 2 e max(1, |log p|).  The entropy is ln z - ln 2 d / z with both
at most ln V + 4 in size (references lie at most 4 below the maximum): e + 2 e
(ln V + 4) <= 2 e (1 + ln V + 4)."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_logprobs import _lib, call  # noqa: E402,F401

pytestmark = pytest.mark.gpu
E = 1e-5


def check(x, ids, k):
    logp, ent, ti, tl = call(x, ids, k)
    d = x.double()
    low = d - d.amax(-1, keepdim=True)                     # no offset: exact in 64 bits
    lz = torch.logsumexp(low, -1, keepdim=True)
    lp = low - lz
    p = lp.exp()
    want = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    off = (ent.double() - want).abs().max()
    assert off <= 2 * E * (5 + math.log(x.shape[1])), float(off)
    top = torch.sort(d, dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ti.long(), top)
    for got, at in ((logp[:, None], ids.long()[:, None]), (tl, top)):
        w = lp.gather(1, at)
        # (a log probability below fp32's range is -inf)
        fits = w > -torch.finfo(torch.float32).max
        err = torch.where(fits, (got.double() - w).abs() / w.abs().clamp(min=1.0), 0.0)
        assert (err <= 2 * E).all(), float(err.max())


@pytest.mark.parametrize("dtype,size,spread", [
    (torch.float32, 0.0, 3.0), (torch.float32, 1e3, 3.0), (torch.float32, 1e5, 1.0), (torch.float32, 9e5, 1.0),
    (torch.float32, 3e6, 4.0), (torch.float32, 1e8, 40.0), (torch.float32, -1e5, 1.0), (torch.float32, -9e5, 1.0),
    (torch.float32, -3e6, 1.0), (torch.bfloat16, 250.0, 3.0), (torch.bfloat16, 3e4, 300.0),
    (torch.bfloat16, 9e5, 9000.0), (torch.bfloat16, -9e5, 9000.0), (torch.float16, 2000.0, 3.0),
    (torch.float16, 3e4, 30.0), (torch.float16, -3e4, 30.0)])
@pytest.mark.parametrize("V", [9, 600, 9001, 100003])
def test_offset_does_not_matter(dtype, size, spread, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(6, V, generator=g, device="cuda") * spread + size).to(dtype)
    x[1, ::3] = -math.inf
    x[1, 1] = size
    x[2] = size                                            # all equal
    ids = torch.randint(0, V, (6,), generator=g, device="cuda").to(torch.int32)
    ids[1] = 1
    check(x, ids, min(V, 5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V", [77, 5003, 66000])
def test_lowest_values_do_not_matter(dtype, V):
    """Masks of the type's lowest value beside ordinary logits, alone, and beside -inf."""
    g = torch.Generator(device="cuda").manual_seed(V)
    big = torch.finfo(dtype).max
    x = (torch.randn(9, V, generator=g, device="cuda") * 3).to(dtype)
    x[0, 5:V - 3] = -big
    x[1, :V // 2] = -big
    x[1, V // 2:V - 2] = -math.inf
    x[2] = -math.inf
    x[2, ::3] = -big                                       # uniform over a third
    x[3] = -big                                            # uniform
    x[4] = -big
    x[4, V // 3] = -big / 2                                # certain
    x[5] = -big / 2
    x[6] = -math.inf
    x[6, V // 2:V // 2 + 3] = 1.0
    x[7, ::2] = -big
    x[8, :V - 1] = -big
    x[8, V - 1] = -100.0
    ids = torch.randint(0, V, (9,), generator=g, device="cuda").to(torch.int32)
    ids[1], ids[2], ids[4], ids[6], ids[7] = V - 1, 3, V // 3, V // 2, 1
    check(x, ids, 3)
