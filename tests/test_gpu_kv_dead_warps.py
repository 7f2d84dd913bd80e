"""Trees and chunks whose rows leave some of a product's four warps without one:
those still take the values past a request's length, and what is not finite, out
of the tiles that the other warps' weights meet."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_kv import BF16, F16, _lib, call, check, make, _spx  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def spoil(s, value):
    """What the cache holds past each request's length, in the pages that it has, and on pages of nobody."""
    spx, (k, v, table) = _spx(), (s["cache"].k, s["cache"].v, s["cache"].block_table)
    page = k.shape[1]
    for b, n in enumerate(s["lens"]):
        if n % page:
            at = int(table[b, n // page])
            k[at, n % page:] = value
            v[at, n % page:] = value


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("rows,heads,kv,D,tree", [
    (17, 4, 4, 128, True), (33, 4, 4, 64, True), (64, 4, 4, 128, True), (40, 16, 16, 64, False), (5, 24, 1, 128, True),
    (129, 4, 4, 128, False), (140, 4, 4, 64, False), (259, 8, 4, 128, False)])
def test_warps_without_rows(rows, heads, kv, D, tree, value, dtype):
    lens = [rows + n for n in (0, 1, 31, 63, 64, 65, 95, 127, 128, 129, 200, 700, 1000, 1537)]
    s = make(lens, [rows] * len(lens), heads=heads, kv=kv, D=D, dtype=dtype, tree=tree, seed=rows)
    spoil(s, value)
    out, lse = call(s)
    check(s, out, lse)
    for _ in range(8):
        again, again_lse = call(s)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
