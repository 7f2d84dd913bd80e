"""The latent-attention, append and log-probability entry points without a GPU:
struct layouts, workspace sizes and every refusal before any CUDA call."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from quantized_expert_gb300 import build, spx
    build.build()
    return spx.load()


@pytest.mark.parametrize("cname,pyname", [("spx_latent_cache", "LatentCacheC"),
                                          ("spx_latent_append_args", "LatentAppendArgs"),
                                          ("spx_latent_args", "LatentArgs"), ("spx_logprobs_args", "LogprobsArgs")])
def test_struct_layouts_match_the_header(tmp_path, cname, pyname):
    from quantized_expert_gb300 import spx
    cls = getattr(spx, pyname)
    fields = [f for f, _ in cls._fields_]
    body = "\n".join(f'    printf("%zu\\n", offsetof({cname}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spx.h"\nint main(void) {\n'
                   f'    printf("%zu\\n", sizeof({cname}));\n' + body + "\n    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got[0] == C.sizeof(cls)
    assert got[1:] == [getattr(cls, f).offset for f in fields]


def cache(**kw):
    from quantized_expert_gb300 import spx
    c = spx.LatentCacheC(spx.SPX_F16, FAKE, 10, 64, 512, 64, 64 * 576, 576, FAKE, 5, 2, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


INV, UNS, WSP = -1, -2, -3
BAD_CACHE = [(dict(cache=None), INV), (dict(block_table=None), INV), (dict(lens=None), INV), (dict(num_pages=0), INV),
             (dict(page_size=0), INV), (dict(page_size=40), UNS), (dict(max_pages=0), INV), (dict(B=0), INV),
             (dict(dtype=2), UNS), (dict(dtype=9), UNS), (dict(R=500), UNS), (dict(R=640), UNS), (dict(R=0), UNS),
             (dict(P=32), UNS), (dict(cache=FAKE + 8), INV), (dict(token_stride=575), INV),
             (dict(token_stride=580), INV), (dict(page_stride=64 * 576 + 4), INV), (dict(page_stride=576), INV)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_cache_refusals(lib, bad, status):
    from quantized_expert_gb300 import spx
    c = cache(**bad)
    a = attention(c)
    assert lib.spx_latent_attention(C.byref(a), None) == status
    b = append(c)
    assert lib.spx_latent_append(C.byref(b), None) == status
    assert spx.status_string(status)


def attention(c, **kw):
    from quantized_expert_gb300 import spx
    a = spx.LatentArgs()
    a.cache, a.N, a.heads, a.q, a.q_start, a.out = C.pointer(c), 3, 16, FAKE, FAKE, FAKE
    a.q_stride, a.out_stride, a.max_q, a.max_len = 16 * 192, 16 * 128, 2, 300
    a.w_uk = a.w_uv = FAKE
    a.dn = a.dv = 128
    a.scale, a.causal, a.ws, a.ws_bytes = 1.0, 1, FAKE, 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(q_start=None), INV), (dict(out=None), INV), (dict(N=-1), INV), (dict(heads=0), INV),
    (dict(max_q=-1), INV), (dict(max_len=-1), INV), (dict(w_uk=None), INV), (dict(w_uv=None), INV),
    (dict(w_uk=None, w_uv=None), INV), (dict(dn=96), UNS), (dict(dv=256, out_stride=16 * 256), UNS),
    (dict(form=3), INV), (dict(form=-1), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(q=FAKE + 2), INV), (dict(out=FAKE + 8), INV),
    (dict(w_uk=FAKE + 8), INV), (dict(q_stride=16 * 192 - 8), INV), (dict(out_stride=16 * 128 - 8), INV),
    (dict(q_stride=16 * 192 + 4), INV), (dict(out_stride=16 * 128 + 1), INV), (dict(ws=None), WSP),
    (dict(ws_bytes=100), WSP), (dict(ws=FAKE + 8), WSP), (dict(heads=2000, q_stride=1 << 30, out_stride=1 << 30), UNS)])
def test_attention_refusals(lib, bad, status):
    c = cache()
    a = attention(c, **bad)
    assert lib.spx_latent_attention(C.byref(a), None) == status
    assert lib.spx_latent_attention(None, None) == INV


def test_attention_without_rows_does_nothing(lib):
    c = cache()
    for kw in (dict(N=0), dict(max_q=0)):
        a = attention(c, **kw)
        assert lib.spx_latent_attention(C.byref(a), None) == 0


def append(c, **kw):
    from quantized_expert_gb300 import spx
    a = spx.LatentAppendArgs()
    a.cache, a.N, a.kv, a.kv_stride, a.req, a.pos, a.w_norm, a.eps = C.pointer(c), 3, FAKE, 576, FAKE, FAKE, FAKE, 1e-6
    a.cos, a.sin, a.max_pos, a.interleaved = FAKE, FAKE, 100, 1
    a.q, a.q_out, a.q_stride, a.q_out_stride, a.heads, a.q_width = FAKE, FAKE, 16 * 192, 16 * 192, 16, 192
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(kv=None), dict(req=None), dict(pos=None), dict(N=-1), dict(kv_stride=568), dict(kv_stride=580),
    dict(kv=FAKE + 8), dict(w_norm=FAKE + 4), dict(cos=None), dict(sin=None), dict(max_pos=0), dict(cos=FAKE + 4),
    dict(q=None), dict(q_out=None), dict(heads=0), dict(q_width=56), dict(q_width=196), dict(q_stride=16 * 192 - 8),
    dict(q_out_stride=16 * 192 + 8), dict(q=FAKE + 8), dict(q_out=FAKE + 8)])
def test_append_refusals(lib, bad):
    a = append(cache(), **bad)
    assert lib.spx_latent_append(C.byref(a), None) == INV
    assert lib.spx_latent_append(None, None) == INV


def test_append_of_nothing(lib):
    a = append(cache(), N=0)
    assert lib.spx_latent_append(C.byref(a), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(logits=None), INV), (dict(N=-1), INV), (dict(V=0), INV), (dict(k=-1), INV), (dict(k=33), UNS),
    (dict(k=8, V=7), INV), (dict(dtype=3), UNS), (dict(stride=999), INV), (dict(ids=None), INV), (dict(logp=None), INV),
    (dict(top_ids=None), INV), (dict(top_logp=None), INV), (dict(k=0), INV), (dict(logits=FAKE + 2), INV)])
def test_logprobs_refusals(lib, bad, status):
    from quantized_expert_gb300 import spx
    a = spx.LogprobsArgs(spx.SPX_F32, FAKE, 1000, 4, 1000, 8, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in bad.items():
        setattr(a, k, v)
    assert lib.spx_token_logprobs(C.byref(a), None) == status
    assert lib.spx_token_logprobs(None, None) == INV


def test_logprobs_of_nothing(lib):
    from quantized_expert_gb300 import spx
    a = spx.LogprobsArgs(spx.SPX_F32, FAKE, 1000, 0, 1000, 8, FAKE, FAKE, FAKE, FAKE, FAKE)
    assert lib.spx_token_logprobs(C.byref(a), None) == 0


def test_workspace_sizes(lib):
    from quantized_expert_gb300 import spx
    size = spx.spx_latent_workspace_size
    assert size(1, 1, 1, 100, 16, dn=128, dv=128) > 0 and size(1, 1, 1, 100, 16) > 0
    for bad in (dict(B=0), dict(N=-1), dict(heads=0), dict(R=100), dict(P=32), dict(dn=128), dict(dv=64),
                dict(dn=96, dv=128), dict(form=7)):
        kw = dict(B=1, N=1, max_q=1, max_len=100, heads=16, R=512, P=64, dn=0, dv=0, form=0)
        kw.update(bad)
        assert size(**kw) == 0, bad
    # a folded call has no expanded form
    assert size(1, 300, 300, 300, 16, form=spx.SPX_LATENT_EXPANDED) == 0
    # more rows, requests and tokens never need less
    last = 0
    for n in (1, 17, 64, 300, 5000):
        now = size(1, n, n, 8000, 16, dn=128, dv=128, form=spx.SPX_LATENT_ABSORBED)
        assert now >= last
        last = now
