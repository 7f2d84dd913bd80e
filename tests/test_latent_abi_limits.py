"""Combinations of arguments that the latent-attention call has to refuse before
any CUDA call, on top of the single refusals."""
import ctypes as C

import pytest

from test_latent_abi import INV, attention, cache, lib  # noqa: F401


@pytest.mark.parametrize("bad", [
    dict(dn=0, dv=0), dict(dn=0), dict(dv=0),                        # weights without widths
    dict(dn=0, dv=0, q_stride=16 * 576, out_stride=16 * 512),        # with the strides of a call without weights
    dict(w_uk=None, w_uv=None, dn=128, dv=0, q_stride=16 * 576, out_stride=16 * 512)])
def test_weights_and_widths_belong_together(lib, bad):  # noqa: F811
    c = cache()
    for form in (0, 1, 2):
        a = attention(c, form=form, **bad)
        assert lib.spx_latent_attention(C.byref(a), None) == INV
