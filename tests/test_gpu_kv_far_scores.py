"""Scores so far from zero that a step of their product with the scale is one or
more (2^23 and beyond, in units of log2): what a row sees best stays its whole
result, and its lse is that score.

Rows count whose best score is ahead of the next by 2^-19 of the sum of its
products' sizes, which no order of fp32 sums (16 partial ones, 2^-22 each) closes,
and by 200, so that the rest weighs nothing.  out is then one value, rounded at
the weight and at the end: 2 u of it.  lse: 2^-18 of that sum."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, U, _lib, call, make, seen_by  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,size", [(F16, 300), (F16, 3000), (F16, 12000), (BF16, 3e4), (BF16, 1e9), (BF16, 1e17)])
@pytest.mark.parametrize("lens,news,heads,kv,D,tree", [
    ([1, 40, 700, 5000], [1, 1, 1, 1], 4, 2, 128, False), ([30000], [1], 8, 1, 64, False), ([900, 64, 2100], [4, 4, 4], 8, 2, 64, False),
    ([4113, 300], [17, 17], 8, 2, 128, True), ([700, 1500, 64], [64, 40, 64], 4, 4, 64, True),
    ([2000, 400], [300, 200], 4, 2, 128, False)])
def test_scores_far_from_zero(lens, news, heads, kv, D, tree, dtype, size):
    s = make(lens, news, heads=heads, kv=kv, D=D, dtype=dtype, tree=tree, seed=D + len(lens))
    s["q"] = (s["q"].float().clamp(-4, 4) * size).to(dtype)
    s["cache"].k.copy_((s["cache"].k.float().clamp(-4, 4) * size).to(dtype))  # (NaN stays)
    s["K"] = [(k.float().clamp(-4, 4) * size).to(dtype) for k in s["K"]]
    out, lse = call(s)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    first, clear = 0, 0
    for b, t in enumerate(s["news"]):
        seen = seen_by(s, b)
        for h in range(heads):
            q, k, v = s["q"][first:first + t, h].double(), s["K"][b][:, h * kv // heads].double(), s["V"][b][:, h * kv // heads]
            score = torch.where(seen, q @ k.T * s["scale"], -math.inf)
            sizes = (q.abs() @ k.abs().T).amax(-1) * s["scale"]
            best, at = score.max(-1)
            rest = score.clone().scatter_(1, at[:, None], -math.inf).amax(-1)
            ok = best - rest > torch.clamp(sizes * 2.0 ** -19, min=200)
            want = v[at].double()
            assert ((out[first:first + t, h].double() - want).abs() <= 2 * U[dtype] * want.abs())[ok].all()
            assert ((lse[first:first + t, h].double() - best).abs() <= sizes * 2.0 ** -18)[ok].all()
            clear += int(ok.sum())
        first += t
    assert clear * 2 >= first * heads
