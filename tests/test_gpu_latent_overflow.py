"""Expanded form: keys and values are written in the type, and one that does not
fit (or is not finite) counts as not finite: rows that see its token show it,
rows that do not keep every bit."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_latent import BF16, F16, _lib, call, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def set_token(s, pos, column, value):
    page = s["cache"].buf.shape[1]
    s["cache"].buf[s["cache"].block_table[0, pos // page].long(), pos % page, column] = value


@pytest.mark.parametrize("lens,news,at", [(700, 300, 650), (700, 300, 513), (130, 130, 127), (130, 130, 129), (512, 257, 511)])
def test_value_beyond_fp16(lens, news, at):
    """v = 120000 is finite in 32 bits and infinite in fp16; its key is an ordinary one."""
    s = make([lens], [news], 4, F16, 64)
    s["w_uk"][:, :, 0] = 0
    s["w_uv"][:, :, 0] = 0
    s["w_uv"][2, 5, 0] = -2.0                              # of one head, in one column
    set_token(s, at, 0, 0.0)
    clean, clean_lse = call(s, form=2)
    assert torch.isfinite(clean).all()
    set_token(s, at, 0, 60000.0)
    out, lse = call(s, form=2)
    first = at - (lens - news)                             # the first row that sees it
    assert torch.equal(out[:first], clean[:first]) and torch.equal(lse[:first], clean_lse[:first])
    others = [0, 1, 3]
    assert torch.equal(out[:, others], clean[:, others])
    assert not torch.isfinite(out[first:, 2, 5]).any()


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_key_beyond_fp16(sign):
    """The same of a key, whether its score rises or falls by it."""
    s = make([300], [100], 2, F16, 64)
    s["w_uk"][:, :, 0] = 0
    s["w_uk"][1, 9, 0] = 2.0
    s["w_uv"][:, :, 0] = 0
    s["q"][:, 1, 9] = sign * 1e-3
    set_token(s, 250, 0, 0.0)
    clean, _ = call(s, form=2)
    set_token(s, 250, 0, 60000.0)
    out, _ = call(s, form=2)
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[:, 0], clean[:, 0])
    assert torch.isnan(out[50:, 1]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_weight_that_is_not_finite_shows(dtype, form, bad):
    s = make([300, 41], [200, 3], 4, dtype, 64)
    clean, _ = call(s, form=form)
    s["w_uv"][1, 7, 9] = bad
    out, _ = call(s, form=form)
    assert not torch.isfinite(out[:, 1, 7]).any()
    others = [0, 2, 3]
    assert torch.equal(out[:, others], clean[:, others])
