"""One speculation step of a small mixture-of-experts decoder: a prompt, K
drafted tokens, their verification and what is accepted.

The layer runs as the library's calls: the new tokens' latent vectors go to the
paged cache (spx_latent_append), attention reads it (spx_latent_attention: the
prompt in the expanded form, drafts and the verify pass in the absorbed one),
the experts follow (spx_moe_layer: INT4 for drafts, FP16 for the verify pass)
and the verify logits are scored (spx_token_logprobs).  Draft and target share
the attention's weights and one cache: the verify pass writes the drafted
positions again, and a rejected token is taken back by a smaller length.

    python examples/speculative_step.py
"""
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np
import torch

import oracle
import spx_workloads as W
from quantized_expert_gb300 import build, spx

HEADS, R, P, NOPE, VALUE, PAGE, VOCAB = 4, 512, 64, 128, 128, 64, 4000


class Decoder:
    """One layer with random weights: the "tiny" expert layer of the tests
    behind latent attention, and a vocabulary."""

    def __init__(self, max_len=1024, seed=0):
        self.s = s = W.CONFIGS["tiny"]
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).half()

        def stack(key, src, view=None):
            a = np.stack([src[e][key] for e in range(s.E)])
            return torch.from_numpy(np.ascontiguousarray(a.view(view) if view is not None else a)).cuda()

        draft = {e: W.gen_w4_expert(s, 0, e) for e in range(s.E)}
        target = {e: oracle.f16_copy_of_w4(draft[e]) for e in range(s.E)}
        self.w4 = spx.spx_w4_repack(stack("qw_gate", draft), stack("s_gate", draft, np.int16), stack("qw_up", draft),
                                    stack("s_up", draft, np.int16), stack("qw_down", draft),
                                    stack("s_down", draft, np.int16))
        self.f16 = spx.spx_f16_repack(*[stack(k, target, np.float16) for k in ("w_gate", "w_up", "w_down")], tc=True)
        self.w_router = torch.from_numpy(W.gen_router(s).view(np.float16)).cuda()
        H = s.H
        self.embed, self.unembed = normal(VOCAB, H, std=1.0), normal(VOCAB, H, std=H ** -0.5)
        self.w_q, self.w_kv = normal(HEADS * (NOPE + P), H, std=H ** -0.5), normal(R + P, H, std=H ** -0.5)
        self.w_o = normal(H, HEADS * VALUE, std=(HEADS * VALUE) ** -0.5)
        self.w_uk, self.w_uv = normal(HEADS, NOPE, R, std=R ** -0.5), normal(HEADS, VALUE, R, std=R ** -0.5)
        self.w_norm = torch.ones(R, dtype=torch.float16, device="cuda")
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, P, 2, device="cuda") / P)
        self.cos, self.sin = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        pages = -(-max_len // PAGE)
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        self.cache = spx.LatentCache(torch.zeros(pages, PAGE, R + P, dtype=torch.float16, device="cuda"), table,
                                     torch.zeros(1, dtype=torch.int32, device="cuda"), R, P)
        self.experts = {}  # workspace and routing buffers by the number of tokens
        # one attention workspace for every call: the larger of the two forms' for the largest call
        size = max(spx.spx_latent_workspace_size(1, max_len, max_len, max_len, HEADS, R, P, NOPE, VALUE, form)
                   for form in (spx.SPX_LATENT_ABSORBED, spx.SPX_LATENT_EXPANDED))
        self.attn_ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def attend(self, x, start):
        """Tokens x [T][H] at the positions start ..: to the cache, then attention over it."""
        T = x.shape[0]
        q = (x @ self.w_q.T).view(T, HEADS, NOPE + P)
        pos = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        args, keep = spx.latent_append_args(self.cache, x @ self.w_kv.T, torch.zeros_like(pos), pos, w_norm=self.w_norm,
                                            cos=self.cos, sin=self.sin, q=q)  # the queries turn in place
        spx.spx_latent_append(args)
        self.cache.lens.fill_(start + T)
        out = torch.empty(T, HEADS, VALUE, dtype=torch.float16, device="cuda")
        rows = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        args, keep = spx.latent_args(q, self.cache, rows, T, start + T, 1 / math.sqrt(NOPE + P), out, self.attn_ws,
                                     w_uk=self.w_uk, w_uv=self.w_uv)
        spx.spx_latent_attention(args)
        return x + out.view(T, -1) @ self.w_o.T

    def mlp(self, x, verify):
        """The expert layer: INT4 experts for drafts, FP16 for the verify pass."""
        s, T = self.s, x.shape[0]
        x = x / x.float().square().mean(-1, keepdim=True).sqrt().half()
        if T not in self.experts:
            self.experts[T] = (spx.new_workspace(T, s.H, s.I, s.E, s.k, 0), spx.Routing.empty(T, s.E, s.k),
                               torch.empty(T, s.E, device="cuda"))
        ws, routing, router = self.experts[T]
        out = torch.empty_like(x)
        args, keep = spx.layer_args(int(verify), x, s.E, s.k, s.renorm, router, routing, out, ws,
                                    w4=None if verify else self.w4, f16=self.f16 if verify else None,
                                    w_router=self.w_router)
        spx.spx_moe_layer(args)
        return x + 0.02 * out

    def logits(self, tokens, start, verify):
        x = self.attend(self.embed[tokens], start)
        return self.mlp(x, verify).float() @ self.unembed.float().T

    def prompt(self, tokens):
        """Only the cache is wanted of a prompt's tokens."""
        self.attend(self.embed[tokens], 0)


def step(model, tokens, K=4):
    """Draft K tokens behind `tokens` (whose last one is not in the cache yet),
    verify them in one pass and return what is accepted with its scores."""
    n = len(tokens) - 1
    drafted, last = [], tokens[-1]
    for i in range(K):
        last = int(model.logits(torch.tensor([last], device="cuda"), n + i, verify=False).argmax())
        drafted.append(last)
    # the verify pass: the last token and the drafted ones, at the same positions
    given = torch.tensor([tokens[-1]] + drafted, device="cuda")
    logits = model.logits(given, n, verify=True)
    # row i scores drafted token i; the last row has none
    wanted = torch.tensor(drafted + [-1], dtype=torch.int32, device="cuda")
    logp, entropy = torch.empty(2, K + 1, device="cuda").unbind()
    top = torch.empty(K + 1, 4, dtype=torch.int32, device="cuda")
    top_logp = torch.empty(K + 1, 4, device="cuda")
    args, keep = spx.logprobs_args(logits, wanted, logp, entropy, top, top_logp)
    spx.spx_token_logprobs(args)
    best = top[:, 0].tolist()
    accepted = 0
    while accepted < K and best[accepted] == drafted[accepted]:
        accepted += 1
    model.cache.lens.fill_(n + 1 + accepted)  # the rejected ones leave the cache
    return dict(drafted=drafted, accepted=accepted, next_token=best[accepted], logp=logp, entropy=entropy, top=top,
                top_logp=top_logp, logits=logits)


def main(prompt_len=300, K=4, steps=3):
    build.build()
    oracle.build()
    spx.load()
    model = Decoder()
    tokens = torch.randint(0, VOCAB, (prompt_len,), generator=torch.Generator().manual_seed(1)).tolist()
    model.prompt(torch.tensor(tokens[:-1], device="cuda"))
    results = []
    for _ in range(steps):
        r = step(model, tokens, K)
        tokens += r["drafted"][:r["accepted"]] + [r["next_token"]]
        results.append(r)
        print("drafted", r["drafted"], "accepted", r["accepted"], "log probabilities",
              [round(v, 2) for v in r["logp"][:K].tolist()], "then", r["next_token"])
    return model, tokens, results


if __name__ == "__main__":
    main()
