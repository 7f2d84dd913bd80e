"""Absorbed form: a latent value that is not finite gives the rows that see its
token what the definition gives them (0 times an infinity is a NaN, also where
the infinity's own score has made the weight 0), and the others nothing."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_latent import BF16, F16, _lib, call, check, make, reference  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("lens,news,at,heads,page,dtype,folded", [
    (200, 9, 195, 16, 64, F16, True), (200, 9, 195, 16, 64, BF16, False), (200, 9, 191, 4, 16, BF16, True),
    (130, 5, 127, 16, 48, F16, True), (130, 5, 128, 20, 64, F16, False), (64, 1, 63, 16, 64, F16, True),
    (65, 2, 3, 16, 64, F16, True), (70, 33, 40, 1, 16, F16, True), (70, 33, 69, 1, 16, F16, True)])
def test_one_latent_value(bad, lens, news, at, heads, page, dtype, folded):
    s = make([lens], [news], heads, dtype, page, folded=folded, seed=at)
    for column in (0, 511, 130):
        s["cache"].buf[s["cache"].block_table[0, at // page].long(), at % page, column] = bad
        s["kv"][0][at, column] = bad
        out, _ = call(s, form=1)
        check(s, (out, None), reference(s))


@pytest.mark.parametrize("bad", [-math.inf, math.nan])
def test_one_rotated_value(bad):
    """A rotated value only makes scores: a row whose score is -inf does without the token."""
    s = make([200], [9], 16, F16, 64, folded=True)
    s["cache"].buf[s["cache"].block_table[0, 195 // 64].long(), 195 % 64, 512] = bad
    s["kv"][0][195, 512] = bad
    out, _ = call(s, form=1)
    check(s, (out, None), reference(s))


@pytest.mark.parametrize("lens,news,heads", [([1], [1], 2), ([40], [3], 16), ([200], [40], 4)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_latent_query_beyond_fp16(lens, news, heads, sign):
    """q W_uk = 120000 in one latent column: finite in 32 bits, not in fp16.  The row
    shows it, also where the infinity's scores are all -inf; no other row does."""
    s = make(lens, news, heads, F16, 64)
    s["cache"].buf[:, :, 5] = -1.0                         # every cached token has the same sign there
    s["w_uk"][1, 3, 5] = 2.0 * sign
    s["w_uk"][1, 3, :5] = 0
    s["w_uk"][1, 3, 6:] = 0
    s["q"][:, 1, 3] = 0
    clean, clean_lse = call(s, form=1)
    s["q"][0, 1, 3] = 60000.0
    out, lse = call(s, form=1)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
