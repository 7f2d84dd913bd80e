"""Alternatives of rows with NaN logits: NaN above everything and ties to the
lower index, also where the NaN is the row's first element, the whole row, or
where every element of the row is asked for.  Indexes have to be equal."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_logprobs import _lib, call  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def order(row):
    x = row.double().tolist()
    return sorted(range(len(x)), key=lambda i: (0, i) if math.isnan(x[i]) else (1, -x[i], i))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("V,k", [(1, 1), (4, 4), (32, 32), (33, 32), (3001, 8), (70000, 20)])
def test_nan_first_everywhere_and_all_asked_for(dtype, V, k):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(5, V, generator=g, device="cuda") * 3).to(dtype)
    x[0, 0] = math.nan
    x[1] = math.nan
    x[2, V - 1] = math.nan
    x[3, 0] = x[3, V // 2] = math.nan
    x[4, 0] = -math.nan  # the sign of a NaN does not matter
    ids = torch.zeros(5, dtype=torch.int32, device="cuda")
    logp, ent, ti, tl = call(x, ids, k)
    assert ti.tolist() == [order(row)[:k] for row in x]
    assert torch.isnan(tl).all() and torch.isnan(logp).all() and torch.isnan(ent).all()
