"""The example keeps one workspace for all its attention calls: its memory does
not grow with the tokens that it decodes."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_speculative_step import example  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_memory_does_not_grow(example):  # noqa: F811
    from quantized_expert_gb300 import build, spx
    build.build()
    spx.load()
    model = example.Decoder()
    tokens = torch.randint(0, example.VOCAB, (200,), generator=torch.Generator().manual_seed(2)).tolist()
    model.prompt(torch.tensor(tokens[:-1], device="cuda"))
    held = []
    for _ in range(5):
        r = example.step(model, tokens, 4)
        tokens += r["drafted"][:r["accepted"]] + [r["next_token"]]
        del r
        torch.cuda.synchronize()
        held.append(torch.cuda.memory_allocated())
    assert held[-1] == held[1], held
