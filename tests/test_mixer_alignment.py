"""Tensors that do not start on 16 bytes: what the kernels take one element at a time is taken
as it is, everything else is a ValueError that names the tensor (the C entry points:
GDN_ERR_ARG).  On the CPU; the C calls' fake pointers are never dereferenced, since each call
is refused for a later reason."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_fwd_amd import abi as A
from gated_deltanet_chunked_fwd_amd import mixer as M
from gated_deltanet_chunked_fwd_amd.binding import lib

BF, F32 = torch.bfloat16, torch.float32


def off(*shape, dtype=BF, by=1):
    """A contiguous tensor that starts `by` elements behind 16 bytes."""
    n = 1
    for s in shape:
        n *= s
    room = torch.zeros(n + 32, dtype=dtype)
    first = -(room.data_ptr() // room.element_size()) % (16 // room.element_size())
    t = room[first + by:first + by + n].view(shape)
    assert t.data_ptr() % 16 == by * t.element_size() % 16
    return t


def args(which, **kw):
    H, n, p = 3, 64, 64
    z = lambda *s, dtype=BF: off(*s, dtype=dtype, by=0)  # noqa: E731
    if which == "conv":
        d, f = dict(x=z(1, 7, 16), weight=z(16, 4), bias=z(16), initial_state=z(1, 3, 16)), M.check_conv_args
    elif which == "conv_step":
        d, f = dict(x=z(3, 16), state=z(5, 3, 16), weight=z(16, 4), bias=z(16)), M.check_conv_step_args
    elif which == "ssm":
        d = dict(x=z(1, 7, H, p), dt=z(1, 7, H), A=z(H, dtype=F32), B=z(1, 7, 1, n), C=z(1, 7, 1, n), initial_state=z(1, H, n, p, dtype=F32))
        f = M.check_ssm_args
    elif which == "ssm_step":
        d = dict(x=z(3, H, p), dt=z(3, H), A=z(H, dtype=F32), B=z(3, 1, n), C=z(3, 1, n), state=z(5, H, n, p, dtype=F32))
        f = M.check_ssm_step_args
    elif which == "delta":
        d = dict(q=z(3, H, n), k=z(3, H, n), v=z(3, H, p), g=z(3, H, dtype=F32), beta=z(3, H), state=z(5, H, n, p, dtype=F32))
        f = M.check_delta_step_args
    else:
        d, f = dict(x=z(6, 4, 32), weight=z(4, 32), bias=z(4, 32), gate=z(6, 4, 32)), M.check_norm_args
    d.update(kw)
    return f(require_cuda=False, **d)


@pytest.mark.parametrize("which,kw", [
    ("conv_step", dict(slots=off(3, dtype=torch.int32))), ("ssm_step", dict(slots=off(3, dtype=torch.int32))),
    ("delta", dict(slots=off(3, dtype=torch.int32, by=3))), ("ssm_step", dict(dt=off(3, 3))), ("ssm", dict(dt=off(1, 7, 3, by=3))),
    ("ssm", dict(A=off(3, dtype=F32), D=off(3, dtype=F32), dt_bias=off(3, dtype=F32))), ("delta", dict(g=off(3, 3, dtype=F32), beta=off(3, 3))),
])
def test_taken(which, kw):
    args(which, **kw)


def test_taken_cu_seqlens_view():
    cu = off(2, dtype=torch.int32)
    cu[1] = 7
    args("conv", cu_seqlens=cu)
    args("ssm", cu_seqlens=cu)


@pytest.mark.parametrize("which,name,t", [
    ("conv", "x", off(1, 7, 16)), ("conv", "weight", off(16, 4)), ("conv", "bias", off(16)), ("conv", "initial_state", off(1, 3, 16)),
    ("conv", "x", off(1, 7, 40, by=0)[..., 4:20]), ("conv_step", "x", off(3, 16)), ("conv_step", "state", off(5, 3, 16)),
    ("ssm", "x", off(1, 7, 3, 64)), ("ssm", "B", off(1, 7, 1, 64)), ("ssm", "C", off(1, 7, 1, 64)),
    ("ssm", "initial_state", off(1, 3, 64, 64, dtype=F32)), ("ssm", "x", off(1, 7, 196, by=0)[..., :192].unflatten(-1, (3, 64))),
    ("ssm_step", "x", off(3, 3, 64)), ("ssm_step", "B", off(3, 1, 64)), ("ssm_step", "state", off(5, 3, 64, 64, dtype=F32)),
    ("ssm_step", "state_out", off(5, 3, 64, 64, dtype=F32)), ("delta", "q", off(3, 3, 64)), ("delta", "state", off(5, 3, 64, 64, dtype=F32)),
    ("norm", "x", off(6, 4, 32)), ("norm", "weight", off(4, 32)), ("norm", "gate", off(6, 4, 32)),
])
def test_refused_by_name(which, name, t):
    with pytest.raises(ValueError, match="^" + name):
        args(which, **{name: t})


def test_workspace_refused():
    ws = off(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="^workspace"):
        M._workspace(ws.device, "gdn_conv_bwd_workspace_bytes", args("conv")[0], ws)


P, INTS, ODD = (ctypes.c_void_p(4096 + k) for k in (0, 4, 2))
BIG = 1 << 31          # slots of a pool that no call takes: the refusal behind the pointers'


def test_entry_points():
    L = lib()
    cs = A.GdnConvShape(B=1, T=1, D=16, W=4, N=BIG, dtype=A.GDN_BF16, param_dtype=A.GDN_BF16, silu=1)
    ss = A.GdnSsmShape(B=1, T=1, H=3, G=1, n=64, p=64, N=BIG, dtype=A.GDN_BF16, dt_dtype=A.GDN_BF16, param_dtype=A.GDN_F32, dt_softplus=1)
    gs = A.GdnShape(B=1, T=1, H=3, dk=64, dv=64, N=BIG, qkv_dtype=A.GDN_BF16, beta_dtype=A.GDN_BF16)
    for slots, want in ((INTS, A.GDN_ERR_UNSUPPORTED), (ODD, A.GDN_ERR_ARG)):
        assert L.gdn_conv_step(P, P, None, P, slots, P, P, ctypes.byref(cs), None) == want
        assert L.gdn_ssm_step(P, P, P, P, P, None, None, P, slots, P, P, ctypes.byref(ss), None) == want
        assert L.gdn_delta_step(P, P, P, P, P, P, slots, 1.0, P, P, ctypes.byref(gs), None) == want
    # dt of bf16 on two bytes, A of fp32 on four; x on sixteen
    assert L.gdn_ssm_step(P, ODD, INTS, P, P, INTS, INTS, P, None, P, P, ctypes.byref(ss), None) == A.GDN_ERR_UNSUPPORTED
    assert L.gdn_ssm_step(P, P, ODD, P, P, None, None, P, None, P, P, ctypes.byref(ss), None) == A.GDN_ERR_ARG
    assert L.gdn_ssm_step(INTS, P, P, P, P, None, None, P, None, P, P, ctypes.byref(ss), None) == A.GDN_ERR_ARG
    assert L.gdn_delta_step(P, P, P, INTS, ODD, P, None, 1.0, P, P, ctypes.byref(gs), None) == A.GDN_ERR_UNSUPPORTED
    assert L.gdn_delta_step(P, P, P, ODD, P, P, None, 1.0, P, P, ctypes.byref(gs), None) == A.GDN_ERR_ARG
    # a prompt: the workspace is the later reason
    sh = A.GdnSsmShape(B=2, T=700, H=3, G=1, n=64, p=64, N=2, dtype=A.GDN_BF16, dt_dtype=A.GDN_BF16, param_dtype=A.GDN_F32,
                       dt_softplus=1, segment_chunks=1)
    for dt, want in ((ODD, A.GDN_ERR_WORKSPACE), (ctypes.c_void_p(4097), A.GDN_ERR_ARG)):
        assert L.gdn_ssm_fwd(P, dt, INTS, P, P, INTS, INTS, None, None, P, None, ctypes.byref(sh), None, 0, None) == want
        assert L.gdn_ssm_bwd(P, dt, INTS, P, P, INTS, INTS, None, None, P, None, P, ODD, INTS, P, P, INTS, INTS, None, ctypes.byref(sh),
                             None, 0, None) == want
    ns = A.GdnNormShape(rows=5, H=2, D=64, dtype=A.GDN_BF16, param_dtype=A.GDN_F32, eps=1e-5)
    for mean, want in ((INTS, A.GDN_ERR_WORKSPACE), (ODD, A.GDN_ERR_ARG)):
        assert L.gdn_norm_bwd(P, P, P, None, mean, mean, P, P, P, P, None, ctypes.byref(ns), None, 0, None) == want
