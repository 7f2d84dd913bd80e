"""Combinations of arguments that the latent-attention call has to refuse before
any CUDA call, on top of the single refusals."""
import ctypes as C

import pytest

from test_latent_abi import INV, UNS, attention, cache, lib  # noqa: F401


@pytest.mark.parametrize("bad", [
    dict(dn=0, dv=0), dict(dn=0), dict(dv=0),                        # weights without widths
    dict(dn=0, dv=0, q_stride=16 * 576, out_stride=16 * 512),        # with the strides of a call without weights
    dict(w_uk=None, w_uv=None, dn=128, dv=0, q_stride=16 * 576, out_stride=16 * 512)])
def test_weights_and_widths_belong_together(lib, bad):  # noqa: F811
    c = cache()
    for form in (0, 1, 2):
        a = attention(c, form=form, **bad)
        assert lib.spx_latent_attention(C.byref(a), None) == INV


@pytest.mark.parametrize("kw,fits", [
    # tiles of 64 tokens times units of rows: B x ceil(max_q x heads / 64) x ceil(max_len / 64), counted in 31 bits
    (dict(B=1024, N=1 << 22, max_q=4096, max_len=1 << 17, heads=16), False),
    (dict(B=64, N=64 * 4096, max_q=4096, max_len=1 << 16, heads=128), True),
    (dict(B=1, N=1 << 20, max_q=1 << 20, max_len=1 << 20, heads=128), False),
    (dict(B=1, N=1 << 14, max_q=1 << 14, max_len=1 << 20, heads=128), True),
    # (only as many rows as there are)
    (dict(B=1, N=17, max_q=1 << 20, max_len=1 << 20, heads=128), True),
    # tokens of the products with the up-projections: 64 a block, 65535 blocks in the grid's third dimension
    (dict(B=1, N=64 * 65535, max_q=1, max_len=100, heads=16, dn=128, dv=128), True),
    (dict(B=1, N=64 * 65535 + 1, max_q=1, max_len=100, heads=16, dn=128, dv=128), False),
    (dict(B=1, N=64 * 65535 + 1, max_q=1, max_len=100, heads=16), True)])
def test_counts_that_do_not_fit_are_refused(lib, kw, fits):  # noqa: F811
    from quantized_expert_gb300 import spx
    assert (spx.spx_latent_workspace_size(form=spx.SPX_LATENT_ABSORBED, **kw) > 0) == fits
    if fits:
        return
    c = cache(B=kw["B"])
    a = attention(c, form=spx.SPX_LATENT_ABSORBED, N=kw["N"], heads=kw["heads"], max_q=kw["max_q"],
                  max_len=kw["max_len"], q_stride=1 << 20, out_stride=1 << 20, ws_bytes=1 << 62)
    if not kw.get("dn"):
        a.w_uk = a.w_uv = None
        a.dn = a.dv = 0
    assert lib.spx_latent_attention(C.byref(a), None) == UNS


def test_one_workspace_serves_every_smaller_call(lib):  # noqa: F811
    from quantized_expert_gb300 import spx
    import random
    rng = random.Random(5)
    for dn in (0, 128):
        most = dict(B=32, N=5000, max_q=3000, max_len=20000, heads=16, dn=dn, dv=dn)
        have = max(spx.spx_latent_workspace_size(form=f, **most) for f in (1, 2))
        for _ in range(3000):
            kw = dict(most, **{k: int(round(most[k] ** rng.random())) for k in ("B", "N", "max_q", "max_len")})
            assert 0 < spx.spx_latent_workspace_size(form=0, **kw) <= have, kw
