"""Acceptance's check that no buffer is named twice, without a GPU: every pair of
places of 128 layers, addresses far apart and side by side."""
import ctypes as C

import pytest

from test_kv_abi import INV, accept, cache, lib  # noqa: F401


@pytest.mark.parametrize("layers", [2, 33, 128])
@pytest.mark.parametrize("step", [16, 4096, 1 << 21, 1 << 32])
def test_a_buffer_named_twice(lib, layers, step):
    from quantized_expert_gb300 import spx
    at = [(1 << 40) + step * i for i in range(2 * layers)]
    places = range(2 * layers) if layers < 128 else [0, 1, 2, 63, 64, 127, 128, 200, 254, 255]
    for i in places:
        for j in places:
            if i == j:
                continue
            twice = list(at)
            twice[i] = at[j]
            assert lib.spx_tree_accept(C.byref(accept(cache(), layers=layers, k=twice[0::2], v=twice[1::2])), None) == INV
    # (none twice: on to the launch, which this machine has no device for)
    ok = accept(cache(), layers=layers, k=at[0::2], v=at[1::2])
    import torch
    if not torch.cuda.is_available():
        assert lib.spx_tree_accept(C.byref(ok), None) == spx.SPX_ERR_CUDA
