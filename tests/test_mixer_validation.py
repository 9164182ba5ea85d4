"""The refusals of gated_deltanet_chunked_fwd_amd.mixer (ValueError before the library is
called) and of its C entry points (an error code before anything is enqueued), on the CPU:
nothing is launched, and the C calls' fake pointers are never dereferenced."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_fwd_amd import abi as A
from gated_deltanet_chunked_fwd_amd import mixer as M
from gated_deltanet_chunked_fwd_amd.binding import lib

BF = torch.bfloat16
Z = torch.zeros


def conv(**kw):
    d = dict(x=Z(2, 7, 16, dtype=BF), weight=Z(16, 4, dtype=BF), bias=Z(16, dtype=BF), initial_state=Z(2, 3, 16, dtype=BF))
    d.update(kw)
    return M.check_conv_args(require_cuda=False, **d)


def test_conv_accepts():
    sh, cu, host = conv()
    assert (sh.B, sh.T, sh.D, sh.W, sh.N, sh.x_stride) == (2, 7, 16, 4, 2, 0) and cu is None and host is None
    conv(weight=Z(16, 4), bias=Z(16))                     # fp32 parameters
    wide = Z(2, 7, 40, dtype=BF)
    assert conv(x=wide[..., 8:24])[0].x_stride == 40
    assert conv(x=wide[:1, :, 8:24], initial_state=None)[0].x_stride == 40
    cu = torch.tensor([0, 3, 3, 7])
    sh, c32, host = conv(x=Z(1, 7, 16, dtype=BF), initial_state=Z(3, 3, 16, dtype=BF), cu_seqlens=cu)
    assert sh.N == 3 and c32.dtype == torch.int32 and host.tolist() == [0, 3, 3, 7]


@pytest.mark.parametrize("kw", [
    dict(x=Z(2, 7, 16, dtype=torch.float16)), dict(x=Z(7, 16, dtype=BF)), dict(x=Z(2, 16, 7, dtype=BF).transpose(1, 2)),
    dict(x=Z(2, 14, 16, dtype=BF)[:, :7]),                # batch rows not T tokens apart
    dict(x=Z(2, 7, 32, dtype=BF)[..., ::2]), dict(weight=Z(16, 5, dtype=BF)), dict(weight=Z(16, 1, dtype=BF)),
    dict(weight=Z(4, 16, dtype=BF)), dict(weight=Z(4, 16, dtype=BF).t()), dict(bias=Z(16)), dict(bias=Z(17, dtype=BF)),
    dict(initial_state=Z(2, 3, 16)), dict(initial_state=Z(2, 4, 16, dtype=BF)), dict(initial_state=Z(1, 3, 16, dtype=BF)),
    dict(cu_seqlens=torch.tensor([0, 7])),                # B = 2
    dict(cu_seqlens_host=torch.tensor([0, 7])),
])
def test_conv_refuses(kw):
    with pytest.raises(ValueError):
        conv(**kw)


@pytest.mark.parametrize("cu", [[0, 8], [1, 7], [0, 5, 4, 7], [0]])
def test_bad_cu_seqlens(cu):
    with pytest.raises(ValueError):
        conv(x=Z(1, 7, 16, dtype=BF), initial_state=None, cu_seqlens=torch.tensor(cu))


def ssm(**kw):
    d = dict(x=Z(2, 7, 4, 64, dtype=BF), dt=Z(2, 7, 4, dtype=BF), A=Z(4), B=Z(2, 7, 2, 128, dtype=BF),
             C=Z(2, 7, 2, 128, dtype=BF), D=Z(4), dt_bias=Z(4), initial_state=Z(2, 4, 128, 64))
    d.update(kw)
    return M.check_ssm_args(require_cuda=False, **d)


def test_ssm_accepts():
    sh = ssm()[0]
    assert (sh.B, sh.T, sh.H, sh.G, sh.n, sh.p, sh.N) == (2, 7, 4, 2, 128, 64, 2)
    ssm(D=None, dt_bias=None, initial_state=None, dt=Z(2, 7, 4))
    whole = Z(2, 7, 4 * 64 + 512, dtype=BF)
    sh = ssm(x=whole[..., :256].unflatten(-1, (4, 64)), B=whole[..., 256:512].unflatten(-1, (2, 128)),
             C=whole[..., 512:].unflatten(-1, (2, 128)))[0]
    assert (sh.x_stride, sh.b_stride, sh.c_stride) == (768, 768, 768)


@pytest.mark.parametrize("kw", [
    dict(x=Z(2, 7, 4, 96, dtype=BF)), dict(x=Z(2, 7, 4, 64)), dict(x=Z(2, 7, 64, 4, dtype=BF).transpose(2, 3)),
    dict(dt=Z(2, 7, 3, dtype=BF)), dict(dt=Z(2, 7, 4, dtype=torch.float16)), dict(A=Z(5)), dict(A=Z(4, dtype=torch.float64)),
    dict(D=Z(4, dtype=BF)), dict(dt_bias=Z(3)), dict(B=Z(2, 7, 3, 128, dtype=BF)), dict(B=Z(2, 7, 2, 32, dtype=BF)),
    dict(C=Z(2, 7, 2, 64, dtype=BF)), dict(C=Z(2, 7, 2, 128)), dict(initial_state=Z(2, 4, 64, 128)),
    dict(initial_state=Z(2, 4, 128, 64, dtype=BF)), dict(segment_chunks=-1),
])
def test_ssm_refuses(kw):
    with pytest.raises(ValueError):
        ssm(**kw)


def steps(which, **kw):
    if which == "conv":
        d = dict(x=Z(3, 16, dtype=BF), state=Z(5, 3, 16, dtype=BF), weight=Z(16, 4, dtype=BF))
        f = M.check_conv_step_args
    elif which == "ssm":
        d = dict(x=Z(3, 4, 64, dtype=BF), dt=Z(3, 4, dtype=BF), A=Z(4), B=Z(3, 2, 64, dtype=BF), C=Z(3, 2, 64, dtype=BF),
                 state=Z(5, 4, 64, 64))
        f = M.check_ssm_step_args
    else:
        d = dict(q=Z(3, 4, 64, dtype=BF), k=Z(3, 4, 64, dtype=BF), v=Z(3, 4, 64, dtype=BF), g=Z(3, 4), beta=Z(3, 4, dtype=BF),
                 state=Z(5, 4, 64, 64))
        f = M.check_delta_step_args
    d.update(kw)
    return f(require_cuda=False, **d)


@pytest.mark.parametrize("which", ["conv", "ssm", "delta"])
def test_steps(which):
    s = Z(5, 3, 16, dtype=BF) if which == "conv" else Z(5, 4, 64, 64)
    sh = steps(which, slots=Z(3, dtype=torch.int32), state=s, state_out=s)
    assert sh.N == 5 and sh.B == 3 and sh.T == 1
    pool = Z(6, *s.shape[1:], dtype=s.dtype)
    for kw in (dict(state=s[:2].clone()),                 # three rows, two states, no slots
               dict(slots=Z(3)), dict(slots=Z(4, dtype=torch.int32)), dict(state=s[:, :1].clone()),
               dict(state=s.double()), dict(state_out=s[:4].clone()), dict(state=pool[:5], state_out=pool[1:])):   # overlapping
        with pytest.raises(ValueError):
            steps(which, **kw)


@pytest.mark.parametrize("kw", [
    dict(q=Z(3, 4, 32, dtype=BF)), dict(k=Z(3, 4, 64)), dict(v=Z(3, 5, 64, dtype=BF)), dict(g=Z(3, 4, dtype=BF)),
    dict(beta=Z(3, 3, dtype=BF)), dict(q=Z(0, 4, 64, dtype=BF)),
])
def test_delta_step_refuses(kw):
    with pytest.raises(ValueError):
        steps("delta", **kw)


def norm(x, **kw):
    return M.check_norm_args(x, require_cuda=False, **kw)


def test_norm():
    sh, stats = norm(Z(6, 4, 32, dtype=BF), weight=Z(4, 32), bias=Z(4, 32), gate=Z(6, 4, 32, dtype=BF))
    assert (sh.rows, sh.H, sh.D) == (6, 4, 32) and tuple(stats) == (6, 4)
    sh, _ = norm(Z(6, 4, 32), weight=Z(32))
    assert (sh.rows, sh.H) == (24, 1)
    x = Z(6, 4, 32, dtype=BF)
    for kw in (dict(weight=Z(3, 32)), dict(weight=Z(4, 31)), dict(weight=Z(32), bias=Z(4, 32)), dict(weight=Z(32), bias=Z(32, dtype=BF)),
               dict(gate=Z(6, 4, 32)), dict(gate=Z(6, 4, 31, dtype=BF)), dict(eps=0.0), dict(eps=float("nan")),
               dict(weight=Z(32, dtype=torch.float16))):
        with pytest.raises(ValueError):
            norm(x, **kw)
    for bad in (Z(32), Z(2, 8193), Z(4, 0), Z(4, 8, dtype=torch.float16), Z(8, 4).t()):
        with pytest.raises(ValueError):
            norm(bad)


def test_outputs_must_not_overlap_inputs():
    x = Z(2, 7, 16, dtype=BF)
    M._check_out(Z(2, 7, 16, dtype=BF), "out", BF, (2, 7, 16), x.device, False, (x, None))
    pool = Z(2 * 7 * 16 + 8, dtype=BF)
    for off, inp in ((0, pool[:224].view(2, 7, 16)), (8, pool[:224].view(2, 7, 16)), (0, pool[16:48])):
        with pytest.raises(ValueError):
            M._check_out(pool[off:off + 224].view(2, 7, 16), "out", BF, (2, 7, 16), x.device, False, (inp,))
    with pytest.raises(ValueError):
        M._check_out(Z(2, 7, 16), "out", BF, (2, 7, 16), x.device, False, ())


# ---- the C entry points ---------------------------------------------------------------------

P = ctypes.c_void_p(4096)
OFF = ctypes.c_void_p(4098)


def conv_shape(**kw):
    d = dict(B=2, T=7, D=16, W=4, N=2, x_stride=0, dtype=A.GDN_BF16, param_dtype=A.GDN_BF16, silu=1)
    d.update(kw)
    return A.GdnConvShape(**d)


def ssm_shape(**kw):
    d = dict(B=2, T=700, H=4, G=2, n=128, p=64, N=2, dtype=A.GDN_BF16, dt_dtype=A.GDN_F32, param_dtype=A.GDN_F32, dt_softplus=1)
    d.update(kw)
    return A.GdnSsmShape(**d)


def norm_shape(**kw):
    d = dict(rows=5, H=2, D=64, dtype=A.GDN_BF16, param_dtype=A.GDN_F32, eps=1e-5)
    d.update(kw)
    return A.GdnNormShape(**d)


def query(name, shape):
    n = ctypes.c_size_t(0)
    return getattr(lib(), name)(ctypes.byref(shape), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(W=5), A.GDN_ERR_UNSUPPORTED), (dict(dtype=3), A.GDN_ERR_UNSUPPORTED), (dict(D=0), A.GDN_ERR_ARG),
    (dict(N=3), A.GDN_ERR_ARG), (dict(x_stride=8), A.GDN_ERR_ARG), (dict(silu=2), A.GDN_ERR_ARG), (dict(T=-1), A.GDN_ERR_ARG),
    (dict(T=1 << 29, B=1, N=1, D=4096), A.GDN_ERR_UNSUPPORTED), (dict(T=1 << 22, B=1, N=1), A.GDN_OK), (dict(D=1 << 27, T=1 << 15), A.GDN_ERR_UNSUPPORTED),
])
def test_conv_shapes_refused(kw, code):
    assert query("gdn_conv_bwd_workspace_bytes", conv_shape(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=32), A.GDN_ERR_UNSUPPORTED), (dict(p=96), A.GDN_ERR_UNSUPPORTED), (dict(G=3), A.GDN_ERR_ARG), (dict(G=0), A.GDN_ERR_ARG),
    (dict(dt_dtype=0), A.GDN_ERR_UNSUPPORTED), (dict(x_stride=4 * 64 + 4), A.GDN_ERR_ARG), (dict(b_stride=128), A.GDN_ERR_ARG),
    (dict(segment_chunks=-1), A.GDN_ERR_ARG), (dict(reserved=1), A.GDN_ERR_ARG), (dict(dt_softplus=2), A.GDN_ERR_ARG),
    (dict(N=1), A.GDN_ERR_ARG),
])
def test_ssm_shapes_refused(kw, code):
    for name in ("gdn_ssm_fwd_workspace_bytes", "gdn_ssm_bwd_workspace_bytes"):
        assert query(name, ssm_shape(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(D=8193), A.GDN_ERR_UNSUPPORTED), (dict(D=0), A.GDN_ERR_ARG), (dict(eps=0.0), A.GDN_ERR_ARG),
    (dict(eps=float("inf")), A.GDN_ERR_ARG), (dict(rows=-1), A.GDN_ERR_ARG), (dict(param_dtype=9), A.GDN_ERR_UNSUPPORTED),
    (dict(rows=1 << 40), A.GDN_ERR_UNSUPPORTED), (dict(reserved=1), A.GDN_ERR_ARG),
])
def test_norm_shapes_refused(kw, code):
    assert query("gdn_norm_bwd_workspace_bytes", norm_shape(**kw))[0] == code


def test_workspaces():
    rc, whole = query("gdn_ssm_fwd_workspace_bytes", ssm_shape(segment_chunks=1000))
    assert rc == 0 and whole == 2 * 11 * 4 * 1024          # the gates of every (chunk, head)
    rc, n = query("gdn_ssm_fwd_workspace_bytes", ssm_shape(segment_chunks=1))
    assert rc == 0 and n >= whole + 2 * 11 * 4 * 128 * 64 * 4   # and a state per (segment, head)
    rc, n = query("gdn_ssm_fwd_workspace_bytes", ssm_shape(T=0))
    assert rc == 0 and n == 0
    rc, n = query("gdn_conv_bwd_workspace_bytes", conv_shape())
    assert rc == 0 and n >= 5 * 16 * 4


def test_entry_points_refuse_before_launch():
    L, big = lib(), ctypes.c_size_t(1 << 40)
    cs, ss, ns = (ctypes.byref(s) for s in (conv_shape(), ssm_shape(), norm_shape()))
    assert L.gdn_conv_fwd(None, P, None, None, None, P, None, cs, None) == A.GDN_ERR_ARG
    assert L.gdn_conv_fwd(P, P, OFF, None, None, P, None, cs, None) == A.GDN_ERR_ARG
    assert L.gdn_conv_fwd(P, P, None, None, P, P, None, cs, None) == A.GDN_ERR_ARG          # cu_seqlens without the host copy
    assert L.gdn_conv_bwd(P, P, None, None, None, P, None, P, P, P, None, cs, P, big, None) == A.GDN_ERR_ARG   # dbias, no bias
    assert L.gdn_conv_bwd(P, P, None, None, None, P, None, P, P, None, None, cs, P, ctypes.c_size_t(8), None) == A.GDN_ERR_WORKSPACE
    assert L.gdn_conv_step(P, P, None, P, None, P, P, cs, None) == A.GDN_ERR_ARG            # T != 1
    one = ctypes.byref(conv_shape(T=1, N=1))
    assert L.gdn_conv_step(P, P, None, P, None, P, P, one, None) == A.GDN_ERR_ARG           # more rows than slots
    assert L.gdn_ssm_fwd(P, P, P, P, P, None, None, None, None, OFF, None, ss, None, 0, None) == A.GDN_ERR_ARG
    split = ctypes.byref(ssm_shape(segment_chunks=1))
    assert L.gdn_ssm_fwd(P, P, P, P, P, None, None, None, None, P, None, split, None, 0, None) == A.GDN_ERR_WORKSPACE
    assert L.gdn_ssm_bwd(*[P] * 5, None, None, None, None, P, None, P, P, None, P, P, None, None, None, ss, P, big, None) == A.GDN_ERR_ARG
    assert L.gdn_ssm_bwd(*[P] * 5, None, None, None, None, P, None, P, P, P, P, P, None, None, None, ss, P, 8, None) == A.GDN_ERR_WORKSPACE
    assert L.gdn_ssm_step(P, P, P, P, P, None, None, P, None, P, P, ss, None) == A.GDN_ERR_ARG
    gs = A.GdnShape(B=2, T=1, H=4, dk=64, dv=64, N=1, qkv_dtype=A.GDN_BF16, beta_dtype=A.GDN_BF16)
    args = [P, P, P, P, P, P, None, 0.1, P, P]
    assert L.gdn_delta_step(*args, ctypes.byref(gs), None) == A.GDN_ERR_ARG                 # more rows than slots
    gs.N, gs.dk = 2, 96
    assert L.gdn_delta_step(*args, ctypes.byref(gs), None) == A.GDN_ERR_UNSUPPORTED
    gs.dk = 64
    assert L.gdn_delta_step(*args[:7], float("nan"), P, P, ctypes.byref(gs), None) == A.GDN_ERR_ARG
    assert L.gdn_norm_fwd(P, None, None, None, OFF, None, None, ns, None) == A.GDN_ERR_ARG
    assert L.gdn_norm_bwd(P, P, P, P, P, P, P, P, P, P, None, ns, P, big, None) == A.GDN_ERR_ARG   # a gate, no dgate
    assert L.gdn_norm_bwd(P, P, P, None, P, P, P, P, P, P, None, ns, None, 0, None) == A.GDN_ERR_WORKSPACE
