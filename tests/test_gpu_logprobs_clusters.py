"""Rows that several blocks of a cluster share, of lengths whose last block has
a short stretch or none: its results reach the first block's memory as early as
they can, over and over."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_logprobs import _lib, call, check  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V", [(torch.float32, 32001), (torch.float32, 32057), (torch.float32, 100004),
                                     (torch.bfloat16, 64003), (torch.bfloat16, 128056), (torch.float16, 130001)])
@pytest.mark.parametrize("N", [1, 17, 31])
def test_short_last_stretches(dtype, V, N):
    g = torch.Generator(device="cuda").manual_seed(V + N)
    x = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    first = call(x, ids, 32)
    check(x, ids, 32, first)
    for _ in range(50):
        assert all(torch.equal(a, b) for a, b in zip(first, call(x, ids, 32)))
