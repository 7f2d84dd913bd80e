"""Values at fp16's largest, as conversions that saturate leave them: a mean of
them is no larger, although rounded weights, each off by 2^-11 at most, may sum to
more than their sum.  Where all of a column is the same value, out lies within
2^-11 of it by the weights and 2^-11 by its own rounding."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import F16, _lib, call, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread", [1, 3, 8])  # of scores: many weights, or few
@pytest.mark.parametrize("lens,news,heads,kv,D,tree", [
    ([2, 40, 517, 2000, 130], [1] * 5, 16, 8, 128, False), ([30000], [1], 8, 2, 64, False), ([900, 64, 2100], [8, 8, 8], 4, 2, 64, False),
    ([700] * 100, [1] * 100, 8, 4, 64, False), ([4113, 300], [17, 17], 8, 2, 128, True), ([700, 1500, 64], [64, 40, 64], 4, 4, 64, True),
    ([60] * 40, [33] * 40, 4, 4, 128, True), ([2000, 400], [300, 200], 4, 2, 128, False), ([3000] * 3, [260] * 3, 8, 2, 64, False),
    ([700] * 60, [64] * 60, 8, 4, 64, False), ([700] * 60, [40] * 60, 8, 4, 128, True)])
def test_a_mean_of_the_largest(lens, news, heads, kv, D, tree, spread):
    s = make(lens, news, heads=heads, kv=kv, D=D, dtype=F16, tree=tree, seed=len(lens))
    s["q"] = s["q"] * spread
    clean, clean_lse = call(s)
    live = ~torch.isnan(s["cache"].v[..., :1])
    for column, value in ((3, 65504.0), (D // 2 + 1, -65504.0), (D - 1, 65504.0)):
        s["cache"].v[..., column:column + 1] = torch.where(live, value, math.nan).half()
    out, lse = call(s)
    assert torch.equal(lse, clean_lse)
    same = [c for c in range(D) if c not in (3, D // 2 + 1, D - 1)]
    assert torch.equal(out[..., same], clean[..., same])
    for column, value in ((3, 65504.0), (D // 2 + 1, -65504.0), (D - 1, 65504.0)):
        assert ((out[..., column].double() - value).abs() <= 65504 * 2.0 ** -10).all(), (out[..., column].isinf().sum(), out.shape)


@pytest.mark.parametrize("rows", [1, 17, 200])
def test_an_infinity_stays_one(rows):
    """One infinity among the largest, where every row sees it: that column alone is not finite."""
    s = make([600 + rows], [rows], heads=4, kv=2, D=64, dtype=F16)
    page = int(s["cache"].block_table[0, 1])
    s["cache"].v[page, 3, 1, 7], s["cache"].v[page, 3, 1, 9] = math.inf, 65504.0
    out, _ = call(s)
    assert torch.isinf(out[:, 2:, 7]).all()
    assert torch.isfinite(out[:, :2]).all() and torch.isfinite(out[:, 2:, 8:]).all()
