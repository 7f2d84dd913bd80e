"""Half of what belongs together is refused by the binding, not left out."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_latent import F16, _lib, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_append_arguments_that_belong_together():
    from quantized_expert_gb300 import spx
    s = make([30], [4], 2, F16, 16)
    kv = torch.zeros(4, 576, dtype=F16, device="cuda")
    at = torch.arange(4, dtype=torch.int32, device="cuda")
    turn = torch.zeros(30, 32, device="cuda")
    for half in (dict(cos=turn), dict(sin=turn), dict(q_out=s["q"])):
        with pytest.raises(ValueError):
            spx.latent_append_args(s["cache"], kv, torch.zeros_like(at), at, **half)
