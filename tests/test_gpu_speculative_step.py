"""The example that runs the append, the attention, the experts and the log
probabilities together: its scores against its own logits, and the cache after
a rejection against a model that never saw the rejected tokens."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_speculative_steps(example):
    K = 4
    model, tokens, results = example.main(prompt_len=300, K=K, steps=3)
    assert sum(r["accepted"] for r in results) > 0  # the draft is the target's own INT4 copy
    for r in results:
        want = torch.log_softmax(r["logits"].double(), -1)
        ids = torch.tensor(r["drafted"], device="cuda")
        assert ((r["logp"][:K].double() - want[:K].gather(1, ids[:, None])[:, 0]).abs() < 1e-4).all()
        assert torch.isnan(r["logp"][K])
        assert torch.equal(r["top"][:, 0].long(), r["logits"].argmax(-1))
        assert ((r["entropy"].double() + (want.exp() * want).sum(-1)).abs() < 1e-4).all()
        assert r["accepted"] == K or r["drafted"][r["accepted"]] != r["next_token"]
    n = int(model.cache.lens[0])
    assert n == len(tokens) - 1
    # the same tokens at once, in another model of the same weights: the same latent vectors in the cache
    # (computed by products of other shapes: fp16 roundings of x W apart, 4 of 2^-11 with a rotation and a norm)
    other = example.Decoder()
    other.prompt(torch.tensor(tokens[:n], device="cuda"))

    def rows(m):
        at = torch.arange(n, device="cuda")
        return m.cache.buf[m.cache.block_table[0, at // example.PAGE].long(), at % example.PAGE].double()

    a, b = rows(model), rows(other)
    assert (a - b).norm() <= 4 * 2.0 ** -11 * b.norm()
