"""The expanded form as a program uses it: in a graph, on a stream of the
caller's, with padded pages, tokens, queries and results; and the log of the
weights' sum of both forms.

lse: the softmax weights' sum is not rounded, so it errs only by the scores'
error.  A score of variance 1 is a sum of products with values rounded once (the
latent queries or the keys), of relative rms u / sqrt(3) each: rms u / sqrt(3)
in all, six deviations 6 u / sqrt(3); fp32 sums 1e-5."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_latent import BF16, F16, U, _lib, call, check, make, reference  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def _spx():
    from quantized_expert_gb300 import spx
    return spx


def test_strides_and_a_stream():
    spx = _spx()
    s = make([517, 130], [300, 129], 3, F16, 48, token_pad=24, page_pad=2)
    N, h = s["q"].shape[:2]
    wide = torch.full((N, h * 192 + 64), math.nan, dtype=F16, device="cuda")
    q = wide[:, 32:32 + h * 192].view(N, h, 192)
    q.copy_(s["q"])
    hold = torch.full((N, h * 128 + 8), 5.0, dtype=F16, device="cuda")
    out = hold[:, 8:].view(N, h, 128)
    ws = torch.zeros(spx.spx_latent_workspace_size(3, N + 50, 400, 900, h, dn=128, dv=128, form=2), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    call(s, form=2, out=out, q=q, ws=ws, stream=stream)
    torch.cuda.synchronize()
    check(s, (out, None), reference(s))
    assert (hold[:, :8] == 5).all()


def test_in_a_graph_with_other_lengths():
    spx = _spx()
    s = make([700, 300], [280, 131], 4, BF16, 64)
    want, _ = call(s, form=2)
    assert torch.equal(call(s, form=2)[0], want)
    out = torch.zeros_like(want)
    ws = spx.new_latent_workspace(s["q"], s["cache"], s["max_q"], s["max_len"], s["w_uk"], s["w_uv"], 2)
    args, keep = spx.latent_args(s["q"], s["cache"], s["q_start"], s["max_q"], s["max_len"], s["scale"], out, ws,
                                 w_uk=s["w_uk"], w_uv=s["w_uv"], form=2)
    spx.spx_latent_attention(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spx.spx_latent_attention(args)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s["cache"].lens[0] = 400                               # lengths are device data
    graph.replay()
    torch.cuda.synchronize()
    s["lens"] = [400, 300]
    s["kv"][0] = s["kv"][0][:400]
    check(s, (out, None), reference(s))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("lens,news,heads", [([517, 65, 1], [17, 1, 1], 16), ([700, 129], [300, 129], 4)])
def test_lse(dtype, form, lens, news, heads):
    s = make(lens, news, heads, dtype, 64, seed=3)
    _, lse = call(s, form=form)
    want = reference(s)[1]
    off = (lse.double() - want).abs().max()
    assert off <= 6 / math.sqrt(3) * U[dtype] + 1e-5, float(off)
