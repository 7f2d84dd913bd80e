"""Scores of key/value attention that are NaN: a query or a key that holds one,
the key as the only token that a warp of the launch for few rows has for a row,
whole or joined from parts.  out and lse of the rows that see it are NaN, in
both launches, and all others as they were."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, _lib, call, make, seen_by  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [1, 4, 16, 17, 64, 200])
@pytest.mark.parametrize("cached", [0, 40, 3000])
def test_a_query_that_is_not_a_number(rows, cached, dtype):
    """One head of one row: that head's out and lse alone."""
    s = make([cached + rows, 33], [rows, 1], heads=4, kv=4, D=64, dtype=dtype)
    clean, clean_lse = call(s)
    row = rows // 2
    s["q"][row, 2, 7] = math.nan
    out, lse = call(s)
    assert torch.isnan(out[row, 2]).all() and torch.isnan(lse[row, 2])
    other = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    other[row, 2] = False
    assert torch.equal(out[other], clean[other]) and torch.equal(lse[other], clean_lse[other])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("length", [1, 17, 33, 49, 113, 129, 145, 2065, 4097, 20001])
@pytest.mark.parametrize("D", [64, 128])
def test_a_lone_key_that_is_not_a_number(length, D, dtype):
    """The newest token: 16 tokens of a tile are a warp's, and here it is alone among them."""
    s = make([length, 700], [1, 1], heads=4, kv=2, D=D, dtype=dtype)
    clean, clean_lse = call(s)
    at = length - 1
    s["cache"].k[int(s["cache"].block_table[0, at // 64]), at % 64, 1, 3] = math.nan
    out, lse = call(s)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(lse[0, :2], clean_lse[0, :2])
    assert torch.equal(out[1], clean[1]) and torch.equal(lse[1], clean_lse[1])


@pytest.mark.parametrize("rows", [2, 16, 17, 64])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("cached", [0, 16, 48, 2048])
def test_a_key_of_the_new_rows(rows, tree, cached):
    """Rows that see the last row's key have a NaN for lse as for out; the others keep their bits."""
    s = make([cached + rows], [rows], heads=2, kv=1, D=64, tree=tree, seed=rows)
    heads = s["heads"]
    clean, clean_lse = call(s)
    bad = cached + rows // 2
    s["cache"].k[int(s["cache"].block_table[0, bad // 64]), bad % 64, 0, 11] = math.nan
    out, lse = call(s)
    seen = seen_by(s, 0)[:, bad]
    assert seen.any() and heads == lse.shape[1]
    assert torch.isnan(out[seen]).all() and torch.isnan(lse[seen]).all()
    assert torch.equal(out[~seen], clean[~seen]) and torch.equal(lse[~seen], clean_lse[~seen])


@pytest.mark.parametrize("rows", [1, 16, 17])
def test_all_keys_not_numbers(rows):
    """No warp has a reference for any row: NaN, and not the sign of a row that sees nothing."""
    s = make([300 + rows], [rows], heads=2, kv=2, D=64)
    s["cache"].k[s["cache"].block_table[0, :5].long()] = math.nan
    out, lse = call(s)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("rows", [1, 16, 17, 64, 200])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_scores_that_are_infinite(rows, value):
    """One value of a key: a score of +inf makes out and lse NaN, one of -inf leaves the token out."""
    s = make([300 + rows], [rows], heads=4, kv=2, D=64)
    clean, clean_lse = call(s)
    at = 150
    s["cache"].k[int(s["cache"].block_table[0, at // 64]), at % 64, 1, 9] = value
    out, lse = call(s)
    assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(lse[:, :2], clean_lse[:, :2])
    up = s["q"][:, 2:, 9] * value > 0
    assert torch.isnan(out[:, 2:][up]).all() and torch.isnan(lse[:, 2:][up]).all()
    down = ~up
    s["cache"].k[int(s["cache"].block_table[0, at // 64]), at % 64, 1] = 0
    # (without the token: its weight taken out of the sum that holds it with a score of 0; two lse, each within 1.3e-4)
    zero, zero_lse = call(s)
    want = torch.log(torch.exp(zero_lse.double()) - 1)[:, 2:][down]
    assert ((lse[:, 2:].double()[down] - want).abs() <= 3e-4).all() and torch.isfinite(out[:, 2:][down]).all()
