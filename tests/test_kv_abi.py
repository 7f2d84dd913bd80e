"""The tree, key/value append and attention entry points without a GPU: struct
layouts, workspace sizes and every refusal before any CUDA call."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned, never dereferenced
INV, UNS, WSP = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from quantized_expert_gb300 import build, spx
    build.build()
    return spx.load()


@pytest.mark.parametrize("cname,pyname", [
    ("spx_kv_cache", "KvCacheC"), ("spx_tree_layout_args", "TreeLayoutArgs"), ("spx_kv_append_args", "KvAppendArgs"),
    ("spx_kv_attention_args", "KvAttentionArgs"), ("spx_tree_accept_args", "TreeAcceptArgs")])
def test_struct_layouts_match_the_header(tmp_path, cname, pyname):
    from quantized_expert_gb300 import spx
    cls = getattr(spx, pyname)
    fields = [f for f, _ in cls._fields_]
    body = "\n".join(f'    printf("%zu\\n", offsetof({cname}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spx.h"\nint main(void) {\n'
                   f'    printf("%zu\\n", sizeof({cname}));\n    printf("%d\\n", SPX_KV_WORKSPACE_ZERO);\n' + body +
                   "\n    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got[0] == C.sizeof(cls) and got[1] == spx.SPX_KV_WORKSPACE_ZERO
    assert got[2:] == [getattr(cls, f).offset for f in fields]


def cache(**kw):
    """8 key heads of 128, pages of 64 tokens, tokens outside heads."""
    from quantized_expert_gb300 import spx
    c = spx.KvCacheC(spx.SPX_F16, FAKE, FAKE + (1 << 24), 10, 64, 8, 128, 64 * 1024, 1024, 128, FAKE, 5, 2, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def layout(**kw):
    from quantized_expert_gb300 import spx
    a = spx.TreeLayoutArgs(2, 3, 2, *[FAKE + 4096 * i for i in range(7)])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append(c, **kw):
    from quantized_expert_gb300 import spx
    a = spx.KvAppendArgs()
    a.cache, a.N, a.k, a.v, a.k_stride, a.v_stride, a.req, a.slot, a.pos = C.pointer(c), 3, FAKE, FAKE, 1024, 1024, FAKE, FAKE, FAKE
    a.q, a.q_out, a.q_stride, a.q_out_stride, a.heads, a.q_norm, a.k_norm, a.eps = FAKE, FAKE, 4096, 4096, 32, FAKE, FAKE, 1e-6
    a.cos, a.sin, a.max_pos, a.P, a.interleaved = FAKE, FAKE, 100, 128, 0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention(c, **kw):
    from quantized_expert_gb300 import spx
    a = spx.KvAttentionArgs()
    a.cache, a.N, a.heads, a.q, a.q_stride, a.out_stride, a.q_start = C.pointer(c), 3, 32, FAKE, 4096, 4096, FAKE
    a.max_q, a.max_len, a.scale, a.causal, a.tree, a.out, a.lse = 2, 300, 0.1, 1, FAKE, FAKE, FAKE
    a.ws, a.ws_bytes = FAKE, 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def accept(c, layers=2, k=None, v=None, **kw):
    from quantized_expert_gb300 import spx
    a = spx.TreeAcceptArgs()
    a.cache, a.n_layers, a.N, a.max_q = C.pointer(c), layers, 3, 2
    n = max(layers, 0)
    a.layer_k = (C.c_void_p * (n + 1))(*(k or [FAKE + 32 * i for i in range(n)]))
    a.layer_v = (C.c_void_p * (n + 1))(*(v or [FAKE + 32 * i + 16 for i in range(n)]))
    for i, f in enumerate(("q_start", "parent", "token", "target", "n_kept", "path", "next", "lens_out")):
        setattr(a, f, FAKE + 4096 * (i + 1))
    for f, x in kw.items():
        setattr(a, f, x)
    return a


BAD_CACHE = [(dict(block_table=None), INV), (dict(lens=None), INV), (dict(num_pages=0), INV), (dict(page_size=0), INV),
             (dict(page_size=40), UNS), (dict(max_pages=0), INV), (dict(B=0), INV), (dict(B=70000), UNS),
             (dict(dtype=2), UNS), (dict(dtype=-1), UNS), (dict(D=96), UNS), (dict(D=0), UNS), (dict(kv_heads=0), INV),
             (dict(kv_heads=2000), UNS), (dict(token_stride=1020), INV), (dict(token_stride=1028), INV),
             (dict(head_stride=120), INV), (dict(head_stride=64), INV), (dict(head_stride=0), INV),
             (dict(page_stride=64 * 1024 - 8), INV), (dict(page_stride=64 * 1024 + 4), INV), (dict(page_stride=-65536), INV),
             (dict(page_stride=1 << 39), UNS)]


@pytest.mark.parametrize("bad,status", BAD_CACHE)
def test_cache_refusals(lib, bad, status):
    c = cache(**bad)
    assert lib.spx_kv_attention(C.byref(attention(c)), None) == status
    assert lib.spx_kv_append(C.byref(append(c)), None) == status
    assert lib.spx_tree_accept(C.byref(accept(c)), None) == status
    assert lib.spx_tree_accept(C.byref(accept(c, layers=0)), None) == status


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(v=FAKE + 2)])
def test_cache_buffers(lib, bad):
    c = cache(**bad)
    assert lib.spx_kv_attention(C.byref(attention(c)), None) == INV
    assert lib.spx_kv_append(C.byref(append(c)), None) == INV


@pytest.mark.parametrize("kw", [
    dict(token_stride=128, head_stride=64 * 128), dict(token_stride=128, head_stride=10 * 64 * 128, page_stride=64 * 128),
    dict(token_stride=2048, page_stride=64 * 2048), dict(kv_heads=1, head_stride=0), dict(num_pages=1, page_stride=0)])
def test_orders_of_the_cache_that_pass(lib, kw):
    c = cache(**kw)
    # (past the cache's own checks, to the next refusal)
    assert lib.spx_kv_attention(C.byref(attention(c, ws=None, heads=32)), None) == WSP


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(q_start=None), INV), (dict(out=None), INV), (dict(N=-1), INV), (dict(heads=0), INV),
    (dict(heads=31), INV), (dict(heads=8 * 65, q_stride=1 << 20, out_stride=1 << 20), UNS), (dict(max_q=-1), INV),
    (dict(max_len=-1), INV), (dict(max_q=65), UNS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(q=FAKE + 2), INV), (dict(out=FAKE + 8), INV),
    (dict(q_stride=4088), INV), (dict(out_stride=4088), INV), (dict(q_stride=4100), INV), (dict(out_stride=4097), INV),
    (dict(ws=None), WSP), (dict(ws_bytes=100), WSP), (dict(ws=FAKE + 8), WSP),
    (dict(tree=None, max_q=1 << 30, N=1 << 30), UNS)])
def test_attention_refusals(lib, bad, status):
    assert lib.spx_kv_attention(C.byref(attention(cache(), **bad)), None) == status
    assert lib.spx_kv_attention(None, None) == INV
    assert lib.spx_kv_attention(C.byref(attention(cache(), cache=None)), None) == INV


def test_attention_without_rows_does_nothing(lib):
    for kw in (dict(N=0), dict(max_q=0), dict(N=0, q=None, out=None)):
        assert lib.spx_kv_attention(C.byref(attention(cache(), **kw)), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(req=None), INV), (dict(slot=None), INV), (dict(N=-1), INV),
    (dict(k_stride=1016), INV), (dict(v_stride=1028), INV), (dict(k=FAKE + 8), INV), (dict(v=FAKE + 8), INV),
    (dict(q_norm=FAKE + 4), INV), (dict(k_norm=FAKE + 4), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(cos=None), INV), (dict(sin=None), INV), (dict(max_pos=0), INV), (dict(cos=FAKE + 4), INV),
    (dict(P=0), UNS), (dict(P=24), UNS), (dict(P=144), UNS), (dict(q=None), INV), (dict(q_out=None), INV),
    (dict(q=None, q_out=None), INV), (dict(heads=0), INV), (dict(q_stride=4088), INV), (dict(q_out_stride=4104), INV),
    (dict(q=FAKE + 8), INV), (dict(q_out=FAKE + 8), INV), (dict(heads=2000, q_stride=1 << 20, q_out_stride=1 << 20), UNS)])
def test_append_refusals(lib, bad, status):
    assert lib.spx_kv_append(C.byref(append(cache(), **bad)), None) == status
    assert lib.spx_kv_append(None, None) == INV


def test_append_wants_two_buffers(lib):
    assert lib.spx_kv_append(C.byref(append(cache(v=FAKE))), None) == INV


def test_append_of_nothing(lib):
    assert lib.spx_kv_append(C.byref(append(cache(), N=0)), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(q_start=None), INV), (dict(lens=None), INV), (dict(B=0), INV), (dict(N=-1), INV), (dict(max_q=-1), INV),
    (dict(max_q=65), UNS), (dict(max_q=65, parent=None), UNS), (dict(max_q=65, mask=None), UNS),
    (dict(slot=FAKE), INV), (dict(pos=FAKE + 4096 * 2 + 8), INV), (dict(mask=FAKE + 4096 * 4 - 16), INV)])
def test_layout_refusals(lib, bad, status):
    assert lib.spx_tree_layout(C.byref(layout(**bad)), None) == status
    assert lib.spx_tree_layout(None, None) == INV


def test_layout_of_nothing(lib):
    for kw in (dict(N=0), dict(max_q=0)):
        assert lib.spx_tree_layout(C.byref(layout(**kw)), None) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(cache=None), INV), (dict(n_layers=-1), INV), (dict(n_layers=129), UNS), (dict(layer_k=None), INV),
    (dict(layer_v=None), INV), (dict(N=-1), INV), (dict(max_q=-1), INV), (dict(max_q=65), UNS), (dict(q_start=None), INV),
    (dict(parent=None), INV), (dict(token=None), INV), (dict(target=None), INV), (dict(n_kept=None), INV),
    (dict(path=None), INV), (dict(next=None), INV), (dict(lens_out=None), INV), (dict(lens_out=FAKE), INV),
    (dict(lens_out=FAKE + 4), INV), (dict(path=FAKE + 4096 * 2), INV), (dict(n_kept=FAKE + 4096 * 8), INV)])
def test_accept_refusals(lib, bad, status):
    assert lib.spx_tree_accept(C.byref(accept(cache(), layers=130 if bad.get("n_layers") == 129 else 2, **bad)),
                               None) == status
    assert lib.spx_tree_accept(None, None) == INV


@pytest.mark.parametrize("kw", [dict(k=[FAKE, None]), dict(v=[None, FAKE]), dict(k=[FAKE, FAKE + 8]),
                                dict(k=[FAKE, FAKE]), dict(k=[FAKE, FAKE + 32], v=[FAKE + 64, FAKE])])
def test_accept_layers(lib, kw):
    assert lib.spx_tree_accept(C.byref(accept(cache(), **kw)), None) == INV


def test_workspace_sizes(lib):
    from quantized_expert_gb300 import spx
    size = spx.spx_kv_workspace_size
    good = dict(B=1, N=1, max_q=1, max_len=100, heads=32, kv_heads=8, D=128)
    assert size(**good) >= spx.SPX_KV_WORKSPACE_ZERO
    for bad in (dict(B=0), dict(B=70000), dict(N=-1), dict(max_q=-1), dict(max_len=-1), dict(heads=0), dict(kv_heads=0),
                dict(heads=33), dict(D=96), dict(heads=8 * 65), dict(N=1 << 30, max_q=1 << 30),
                dict(B=60000, N=1 << 20, max_q=1 << 20, max_len=1 << 30)):
        assert size(**{**good, **bad}) == 0, bad
    # no fewer bytes for more rows, requests and tokens
    last = 0
    for n in (1, 4, 17, 64, 300, 5000):
        now = size(2, n, n, 8000, 32, 8)
        assert now >= last
        last = now


@pytest.mark.parametrize("bad,status", [
    (dict(scale=3e38), INV),  # its product with log2(e) is infinite
    (dict(max_len=0x7fffffff), UNS), (dict(max_len=0x7fff0001), UNS)])
def test_attention_beyond_what_is_counted(lib, bad, status):
    c = cache(max_pages=1 << 25)  # 2^31 tokens
    assert lib.spx_kv_attention(C.byref(attention(c, N=1, max_q=1, tree=None, **bad)), None) == status


@pytest.mark.parametrize("bad", [dict(num_pages=0x7fffffff, page_stride=1 << 37), dict(token_stride=1 << 30, num_pages=1 << 20,
                                                                                       page_stride=1 << 36)])
def test_caches_larger_than_any_memory(lib, bad):
    c = cache(**bad)
    assert lib.spx_kv_attention(C.byref(attention(c)), None) == UNS
    assert lib.spx_kv_append(C.byref(append(c)), None) == UNS
    assert lib.spx_tree_accept(C.byref(accept(c)), None) == UNS
