"""Sizes that the mixer's entry points take and refuse for their launches' workgroups (at most
2^32 - 1 work-items a launch); on the CPU, nothing is launched."""
import ctypes

import pytest

from gated_deltanet_chunked_fwd_amd import abi as A
from gated_deltanet_chunked_fwd_amd.binding import lib


def norm(**kw):
    d = dict(rows=5, H=1, D=64, dtype=A.GDN_BF16, param_dtype=A.GDN_F32, eps=1e-5)
    d.update(kw)
    n = ctypes.c_size_t(0)
    sh = A.GdnNormShape(**d)
    rc = lib().gdn_norm_bwd_workspace_bytes(ctypes.byref(sh), ctypes.byref(n))
    if rc == A.GDN_OK:                       # then the forward pass takes it too: it misses its tensors only
        assert lib().gdn_norm_fwd(None, None, None, None, None, None, None, ctypes.byref(sh), None) == A.GDN_ERR_ARG
    else:
        assert lib().gdn_norm_fwd(None, None, None, None, None, None, None, ctypes.byref(sh), None) == rc
    return rc


@pytest.mark.parametrize("kw,code", [
    (dict(rows=1 << 20, H=16, D=128), A.GDN_OK),             # 16 lanes a row: 2^20 workgroups
    (dict(rows=1 << 19, H=32, D=64), A.GDN_OK),
    (dict(rows=(1 << 24) + 1, D=64), A.GDN_OK),
    (dict(rows=1 << 28, H=1, D=64), A.GDN_OK),               # 8 lanes, 2^23 workgroups
    (dict(rows=1 << 29, H=1, D=64), A.GDN_ERR_UNSUPPORTED),
    (dict(rows=(1 << 24) - 1, D=8192), A.GDN_OK),            # a workgroup a row
    (dict(rows=1 << 24, D=8192), A.GDN_ERR_UNSUPPORTED),
    (dict(rows=1 << 62, H=3), A.GDN_ERR_UNSUPPORTED),
    (dict(rows=1, H=1 << 20, D=8192), A.GDN_ERR_UNSUPPORTED),   # 2^34 columns of weights' gradients
])
def test_norm(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("D,code", [(1 << 24, A.GDN_OK), (1 << 26, A.GDN_ERR_UNSUPPORTED)])
def test_convolution_gradients_of_many_channels(D, code):
    """(W + 1) D columns of sums."""
    sh = A.GdnConvShape(B=1, T=1, D=D, W=4, N=1, dtype=A.GDN_BF16, param_dtype=A.GDN_BF16, silu=1)
    n = ctypes.c_size_t(0)
    assert lib().gdn_conv_bwd_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == code
