"""Waits of the latent-attention launches: none of them runs out in calls whose
units have one, two, three or many tiles, while another stream keeps the SMs'
issue slots and caches busy."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_latent import BF16, F16, _lib, call, check, make, reference  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,news,heads,dtype", [
    ([64 * t + 1 for t in range(1, 40)], [1] * 39, 16, F16), ([63, 65, 129, 191, 400, 1000] * 8, [2] * 48, 16, BF16),
    ([100, 150, 250, 350, 900] * 9, [5] * 45, 16, F16), ([5000], [1], 16, F16), ([20000], [4], 16, BF16)])
def test_no_wait_runs_out(lens, news, heads, dtype):
    s = make(lens, news, heads, dtype, 64, seed=len(lens))
    first, _ = call(s, form=1)
    check(s, (first, None), reference(s))
    other, noise = torch.cuda.Stream(), torch.randn(1 << 22, device="cuda")
    for _ in range(60):
        with torch.cuda.stream(other):
            for _ in range(4):
                noise.mul_(1.0001).sin_()
        # (call() asserts that the workspace's status is clean)
        assert torch.equal(call(s, form=1, wait_budget_ns=1_000_000_000)[0], first)
