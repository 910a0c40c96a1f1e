"""Sizes of the layer norm on the host: rows are only counted, up to 2^40 elements in all."""
import ctypes

import pytest

from float8linear_tensorwise_amax_amd import f8lin

lib = f8lin._lib
EINVAL, ESHAPE = 1, 2


@pytest.mark.parametrize("rows,cols,status", [((1 << 22) + 1, 64, EINVAL), (1 << 38, 4, EINVAL), (1 << 40, 0, EINVAL),
                                              ((1 << 38) + 1, 4, ESHAPE), ((1 << 40) + 1, 1, ESHAPE), (1 << 62, 0, ESHAPE),
                                              (1 << 62, 4, ESHAPE), (5, (1 << 22) + 1, ESHAPE), (1 << 18, 1 << 22, EINVAL)])
def test_rows(rows, cols, status):
    """(No tensor is given: a size that is allowed fails for that, and nothing is launched; no column, no data: eps.)"""
    fwd = f8lin.LayerNormFwdArgs(rows=rows, cols=cols, eps=-1.0)
    assert lib.f8lin_layer_norm_forward(ctypes.byref(fwd), None) == status
    if cols:
        bwd = f8lin.LayerNormBwdArgs(rows=rows, cols=cols, dx=64)
        assert lib.f8lin_layer_norm_backward(ctypes.byref(bwd), None) == status
        assert (lib.f8lin_layer_norm_workspace_bytes(rows, cols) > 0) == (status == EINVAL)
