"""Binding of the operators around the delta rule (include/gdn.h): the short causal
convolution, the selective state space scan, the norm of the heads' outputs and the
single-token steps.

Argument checking and marshalling only, like ``binding``: a wrong type, shape, layout or
device raises ValueError before the library is called.  Tensors start on 16 bytes, but those
that the kernels take one element at a time: cu_seqlens, slots, g, beta, dt, A, D, dt_bias, mean
and rstd may start anywhere.  Calls run on the current stream
of the tensors' device, allocate their outputs and workspace there and return without
waiting; a workspace or output that the caller passes belongs to one call at a time.
They can be captured into a graph if cu_seqlens comes with its host copy.
"""
import ctypes
import math

import torch

from .abi import GDN_BF16, GDN_F32, GDN_OK, GdnConvShape, GdnNormShape, GdnShape, GdnSsmShape
from .binding import GdnError, lib

_TYPES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
_F32 = (torch.float32,)
_FP = (torch.bfloat16, torch.float32)


def _fail(what):
    raise ValueError(what)


def _check(t, name, dtypes, shape, device, cuda, align=16):
    """A contiguous tensor of one of the types and the shape, on the device, that starts on
    `align` bytes (1: on an element)."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.device == device and
            t.is_contiguous() and (t.is_cuda or not cuda) and t.data_ptr() % align == 0):
        return
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        _fail("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if t.shape != shape:
        _fail("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != device:
        _fail("%s is on %s, expected %s" % (name, t.device, device))
    if cuda and not t.is_cuda:
        _fail("%s must be a device tensor" % name)
    if not t.is_contiguous():
        _fail("%s must be contiguous" % name)
    _fail("%s must start on a multiple of %d bytes (a copy does)" % (name, align))


def _check_tokens(t, name, dtypes, shape, device, cuda):
    """Token-major [B, T, ...]: contiguous, or a slice of a wider contiguous tensor (each
    token's elements contiguous, tokens evenly apart).  Returns the token stride."""
    if not isinstance(t, torch.Tensor):
        _fail("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        _fail("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if t.shape != shape:
        _fail("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if device is not None and t.device != device:
        _fail("%s is on %s, expected %s" % (name, t.device, device))
    if cuda and not t.is_cuda:
        _fail("%s must be a device tensor" % name)
    if t.data_ptr() % 16:
        _fail("%s must start on a multiple of 16 bytes (a copy does)" % name)
    if t.is_contiguous():
        return 0
    B, T = shape[:2]
    width = 1
    for n, st in zip(reversed(shape[2:]), reversed(t.stride()[2:])):
        if n != 1 and st != width:
            _fail("%s: the elements of a token must be contiguous" % name)
        width *= n
    stride = t.stride(1) if T > 1 else t.stride(0) if B > 1 else width
    if stride < width or (B > 1 and t.stride(0) != T * stride):
        _fail("%s must be contiguous, or a slice of the last axes of a contiguous tensor" % name)
    return stride


def _span(t):
    """The addresses from a tensor's first to behind its last element."""
    at, n = t.data_ptr(), t.numel()
    if n == 0 or t.is_contiguous():
        return at, at + n * t.element_size()
    return at, at + (sum((n - 1) * st for n, st in zip(t.shape, t.stride())) + 1) * t.element_size()


def _check_out(t, name, dtype, shape, device, cuda, inputs):
    """A caller's output buffer (None is allowed), which no input may share memory with."""
    if t is None:
        return
    _check(t, name, (dtype,), shape, device, cuda)
    lo, hi = _span(t)
    for u in inputs:
        if u is not None:
            a, b = _span(u)
            if a < hi and lo < b:
                _fail("%s must not overlap an input" % name)


def _sequences(B, T, cu, host, device, cuda):
    """(N, int32 device cu_seqlens, host copy as the C ABI reads it)."""
    if cu is None:
        if host is not None:
            _fail("cu_seqlens_host given without cu_seqlens")
        return B, None, None
    if B != 1:
        _fail("packed sequences (cu_seqlens) need B == 1")
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.numel() < 2:
        _fail("cu_seqlens must be a 1-D tensor of N + 1 offsets")
    N = cu.numel() - 1
    _check(cu, "cu_seqlens", (torch.int32, torch.int64), (N + 1,), device, cuda, 1)
    if host is None:
        host = cu.to("cpu")
    elif not (isinstance(host, torch.Tensor) and not host.is_cuda and tuple(host.shape) == (N + 1,) and
              host.dtype in (torch.int32, torch.int64)):
        _fail("cu_seqlens_host must be a host int32/int64 tensor of N + 1 offsets")
    host = host.to(torch.int32).contiguous()
    if N <= 64:                              # (a list is quicker up to some 200)
        at = host.tolist()
        fine = at[0] == 0 and at[-1] == T and all(a <= b for a, b in zip(at, at[1:]))
    else:
        fine = int(host[0]) == 0 and int(host[-1]) == T and not bool((host[1:] < host[:-1]).any())
    if not fine:
        _fail("cu_seqlens must start at 0, never fall and end at T")
    return N, cu.to(torch.int32), host


def _host_ptr(host):
    return None if host is None else ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_int32))


def _p(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without the Stream object around it (a decode step's call is
# a few microseconds in all, and the object two of them).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, what, *args):
    """Calls an entry point, its last argument the current stream of the device."""
    f = getattr(lib(), what)
    if device.index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            rc = f(*args, _raw_stream(device.index))
    if rc != GDN_OK:
        raise GdnError(rc, what)


def _need_bytes(device, what, shape):
    """The workspace size that a query reports for a shape, with the device current (the
    split of a scan goes by its CUs)."""
    n = ctypes.c_size_t(0)
    f = getattr(lib(), what)
    if device.index == torch.cuda.current_device():
        rc = f(ctypes.byref(shape), ctypes.byref(n))
    else:
        with torch.cuda.device(device):
            rc = f(ctypes.byref(shape), ctypes.byref(n))
    if rc != GDN_OK:
        raise GdnError(rc, what)
    return n.value


def _workspace(device, what, shape, workspace):
    """(workspace or None, bytes): the caller's if it is large enough, else a new one."""
    if workspace is not None and not (isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8 and
                                      workspace.dim() == 1 and workspace.is_contiguous() and workspace.device == device and
                                      workspace.data_ptr() % 16 == 0):
        _fail("workspace must be a contiguous 1-D uint8 tensor on the inputs' device that starts on a multiple of 16 bytes")
    need = _need_bytes(device, what, shape)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    return workspace, 0 if workspace is None else workspace.numel()


# ---- short convolution ----------------------------------------------------------------

def check_conv_args(x, weight, bias=None, initial_state=None, cu_seqlens=None, cu_seqlens_host=None, silu=True,
                    require_cuda=True):
    """Checks the convolution's inputs; returns (GdnConvShape, int32 cu_seqlens, host copy)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        _fail("x must be a 3-D tensor [B, T, D]")
    B, T, D = x.shape
    if B < 1 or D < 1:
        _fail("x has shape %s: B and D must be at least 1" % (tuple(x.shape),))
    stride = _check_tokens(x, "x", _FP, (B, T, D), None, require_cuda)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        _fail("weight must be a 2-D tensor [D, W]")
    W = weight.shape[1]
    _check(weight, "weight", _FP, (D, W), x.device, require_cuda)
    if bias is not None:
        _check(bias, "bias", (weight.dtype,), (D,), x.device, require_cuda)
    N, cu, host = _sequences(B, T, cu_seqlens, cu_seqlens_host, x.device, require_cuda)
    if not 2 <= W <= 4:
        _fail("weight must have 2, 3 or 4 taps")
    if initial_state is not None:
        _check(initial_state, "initial_state", (x.dtype,), (N, W - 1, D), x.device, require_cuda)
    return GdnConvShape(B, T, D, W, N, stride, _TYPES[x.dtype], _TYPES[weight.dtype], int(bool(silu)),
                        _host_ptr(host)), cu, host


def conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, cu_seqlens_host=None, silu=True,
             output_final_state=True, out=None):
    """Short causal convolution of x [B, T, D] with weight [D, W] (W 2..4) and bias [D], then
    SiLU.  Returns ``(y, final_state)``; the states are the last W - 1 inputs of each
    sequence, [N, W - 1, D], oldest first (initial_state None: zero).  x may be a slice of a
    wider tensor's last axis."""
    sh, cu, host = check_conv_args(x, weight, bias, initial_state, cu_seqlens, cu_seqlens_host, silu)
    _check_out(out, "out", x.dtype, x.shape, x.device, True, (x, weight, bias, initial_state))
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fin = torch.empty((sh.N, sh.W - 1, sh.D), dtype=x.dtype, device=x.device) if output_final_state else None
    _call(x.device, "gdn_conv_fwd", _p(x), _p(weight), _p(bias), _p(initial_state), _p(cu), _p(y), _p(fin),
          ctypes.byref(sh))
    return y, fin


def conv_bwd(x, weight, bias, dy, initial_state=None, d_final_state=None, cu_seqlens=None, cu_seqlens_host=None,
             silu=True, want_d_initial_state=True, workspace=None):
    """Gradients of <dy, y> + <d_final_state, final_state> of conv_fwd.  Returns ``(dx,
    dweight, dbias, d_initial_state)`` (dbias None without a bias, the last None unless
    wanted), in the types of what they belong to."""
    sh, cu, host = check_conv_args(x, weight, bias, initial_state, cu_seqlens, cu_seqlens_host, silu)
    _check(dy, "dy", (x.dtype,), x.shape, x.device, True)
    states = (sh.N, sh.W - 1, sh.D)
    if d_final_state is not None:
        _check(d_final_state, "d_final_state", (x.dtype,), states, x.device, True)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    di = torch.empty(states, dtype=x.dtype, device=x.device) if want_d_initial_state else None
    ws, nb = _workspace(x.device, "gdn_conv_bwd_workspace_bytes", sh, workspace)
    _call(x.device, "gdn_conv_bwd", _p(x), _p(weight), _p(bias), _p(initial_state), _p(cu), _p(dy), _p(d_final_state),
          _p(dx), _p(dw), _p(db), _p(di), ctypes.byref(sh), _p(ws), nb)
    return dx, dw, db, di


def _check_slots(state, state_out, slots, R, shape, dtype, device, cuda):
    """The pool of states, its output and the rows' slots of a single-token step."""
    if not isinstance(state, torch.Tensor) or state.dim() != len(shape) + 1 or state.shape[0] < 1:
        _fail("state must be a tensor [S, %s]" % ", ".join(str(n) for n in shape))
    S = state.shape[0]
    _check(state, "state", (dtype,), (S,) + shape, device, cuda)
    if state_out is not None and state_out is not state:
        _check(state_out, "state_out", (dtype,), (S,) + shape, device, cuda)
        apart = abs(state_out.data_ptr() - state.data_ptr())
        if apart != 0 and apart < state.numel() * state.element_size():
            _fail("state_out must be state itself or not overlap it")
    if slots is not None:
        _check(slots, "slots", (torch.int32,), (R,), device, cuda, 1)
    elif R > S:
        _fail("%d rows need slots, or as many states (there are %d)" % (R, S))
    return S


def check_conv_step_args(x, state, weight, bias=None, slots=None, state_out=None, silu=True, require_cuda=True):
    """Checks conv_step's arguments; returns the GdnConvShape."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.numel() < 1:
        _fail("x must be a 2-D tensor [R, D] with R, D >= 1")
    R, D = x.shape
    _check(x, "x", _FP, (R, D), x.device, require_cuda)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or not 2 <= weight.shape[1] <= 4:
        _fail("weight must be a 2-D tensor [D, W] with 2, 3 or 4 taps")
    W = weight.shape[1]
    _check(weight, "weight", _FP, (D, W), x.device, require_cuda)
    if bias is not None:
        _check(bias, "bias", (weight.dtype,), (D,), x.device, require_cuda)
    S = _check_slots(state, state_out, slots, R, (W - 1, D), x.dtype, x.device, require_cuda)
    return GdnConvShape(R, 1, D, W, S, 0, _TYPES[x.dtype], _TYPES[weight.dtype], int(bool(silu)), None)


def conv_step(x, state, weight, bias=None, slots=None, state_out=None, silu=True, out=None):
    """conv_fwd for one token of each of R rows: x [R, D], state [S, W - 1, D].  Returns y.

    Row i continues the state slots[i] (or i).  The state is updated in place, or written
    to state_out (only the slots in use).  Rows with the same slot are applied in order; a
    slot outside [0, S) is padding: y is zero there and no state is touched."""
    sh = check_conv_step_args(x, state, weight, bias, slots, state_out, silu)
    _check_out(out, "out", x.dtype, x.shape, x.device, True, (x, weight, bias, state, state_out))
    y = out if out is not None else torch.empty_like(x)
    _call(x.device, "gdn_conv_step", _p(x), _p(weight), _p(bias), _p(state), _p(slots), _p(y),
          _p(state if state_out is None else state_out), ctypes.byref(sh))
    return y


# ---- selective scan -------------------------------------------------------------------

def _check_params(A, D, dt_bias, H, device, cuda):
    if not isinstance(A, torch.Tensor):
        _fail("A must be a torch.Tensor")
    _check(A, "A", _FP, (H,), device, cuda, 1)
    for t, name in ((D, "D"), (dt_bias, "dt_bias")):
        if t is not None:
            _check(t, name, (A.dtype,), (H,), device, cuda, 1)


def check_ssm_args(x, dt, A, B, C, D=None, dt_bias=None, initial_state=None, cu_seqlens=None, cu_seqlens_host=None,
                   dt_softplus=True, segment_chunks=0, require_cuda=True):
    """Checks the scan's inputs; returns (GdnSsmShape, int32 cu_seqlens, host copy)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        _fail("x must be a 4-D tensor [B, T, H, p]")
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        _fail("B must be a 4-D tensor [B, T, G, n]")
    nb, T, H, p = x.shape
    G, n = B.shape[2:]
    dev = x.device
    if nb < 1 or H < 1:
        _fail("x has shape %s: B and H must be at least 1" % (tuple(x.shape),))
    if G < 1 or H % G:
        _fail("the groups of B (%d) must divide the heads of x (%d)" % (G, H))
    if n not in (64, 128) or p not in (64, 128):
        _fail("state size %d and head size %d must be 64 or 128" % (n, p))
    xs = _check_tokens(x, "x", _FP, (nb, T, H, p), None, require_cuda)
    bs = _check_tokens(B, "B", (x.dtype,), (nb, T, G, n), dev, require_cuda)
    cs = _check_tokens(C, "C", (x.dtype,), (nb, T, G, n), dev, require_cuda)
    for t, st, name in ((x, xs, "x"), (B, bs, "B"), (C, cs, "C")):
        if st * t.element_size() % 16:
            _fail("%s: tokens %d elements apart, must be a multiple of 16 bytes" % (name, st))
    _check(dt, "dt", _FP, (nb, T, H), dev, require_cuda, 1)
    _check_params(A, D, dt_bias, H, dev, require_cuda)
    N, cu, host = _sequences(nb, T, cu_seqlens, cu_seqlens_host, dev, require_cuda)
    if initial_state is not None:
        _check(initial_state, "initial_state", _F32, (N, H, n, p), dev, require_cuda)
    if not 0 <= segment_chunks < 2 ** 31:
        _fail("segment_chunks must be from 0 to 2^31 - 1")
    return GdnSsmShape(nb, T, H, G, n, p, N, xs, bs, cs, _TYPES[x.dtype], _TYPES[dt.dtype], _TYPES[A.dtype],
                       int(bool(dt_softplus)), segment_chunks, 0, _host_ptr(host)), cu, host


def ssm_fwd(x, dt, A, B, C, D=None, dt_bias=None, initial_state=None, cu_seqlens=None, cu_seqlens_host=None,
            dt_softplus=True, output_final_state=True, out=None, workspace=None, segment_chunks=0):
    """Selective state space scan: with delta = softplus(dt + dt_bias),

        h_t = exp(delta_t A) h_{t-1} + delta_t B_t x_t^T,    y_t = C_t h_t + D x_t

    x [B, T, H, p]; dt [B, T, H]; A, D, dt_bias [H]; B, C [B, T, G, n], shared by the H / G heads
    of a group; n, p 64 or 128.  Returns ``(y, final_state)``, states [N, H, n, p] fp32
    (initial_state None: zero).  x, B and C may be slices of a wider tensor.
    segment_chunks > 0 sets the length, in chunks of 64 tokens, of the segments that a
    sequence is split into (0: chosen so that they fill the GPU).

    bf16 outputs come from the state as bf16 pairs (17 bits); the state itself is carried in fp32.
    No output depends on later tokens, whatever their values; an infinity in x may come out as NaN
    in its column of the states and of later outputs."""
    sh, cu, host = check_ssm_args(x, dt, A, B, C, D, dt_bias, initial_state, cu_seqlens, cu_seqlens_host, dt_softplus,
                                  segment_chunks)
    _check_out(out, "out", x.dtype, x.shape, x.device, True, (x, dt, A, B, C, D, dt_bias, initial_state))
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fin = torch.empty((sh.N, sh.H, sh.n, sh.p), dtype=torch.float32, device=x.device) if output_final_state else None
    ws, nb = _workspace(x.device, "gdn_ssm_fwd_workspace_bytes", sh, workspace)
    _call(x.device, "gdn_ssm_fwd", _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(initial_state), _p(cu),
          _p(y), _p(fin), ctypes.byref(sh), _p(ws), nb)
    return y, fin


def ssm_bwd(x, dt, A, B, C, D, dt_bias, dy, initial_state=None, d_final_state=None, cu_seqlens=None,
            cu_seqlens_host=None, dt_softplus=True, want_d_initial_state=True, workspace=None, segment_chunks=0):
    """Gradients of <dy, y> + <d_final_state, final_state> of ssm_fwd.  Returns ``(dx, ddt, dA,
    dB, dC, dD, ddt_bias, d_initial_state)``, in the types of what they belong to (dD and
    ddt_bias None without D and dt_bias, the last None unless wanted).  Segments are of at most 16
    chunks.  A value that is NaN or infinite reaches the gradients of its whole chunk of 64 tokens,
    and ddt and the parameters' of its sequence."""
    sh, cu, host = check_ssm_args(x, dt, A, B, C, D, dt_bias, initial_state, cu_seqlens, cu_seqlens_host, dt_softplus,
                                  segment_chunks)
    dev = x.device
    _check(dy, "dy", (x.dtype,), x.shape, dev, True)
    states = (sh.N, sh.H, sh.n, sh.p)
    if d_final_state is not None:
        _check(d_final_state, "d_final_state", _F32, states, dev, True)
    dx, ddt, dA = torch.empty(x.shape, dtype=x.dtype, device=dev), torch.empty_like(dt), torch.empty_like(A)
    dB, dC = (torch.empty(B.shape, dtype=x.dtype, device=dev) for _ in range(2))
    dD = None if D is None else torch.empty_like(D)
    dbias = None if dt_bias is None else torch.empty_like(dt_bias)
    dh = torch.empty(states, dtype=torch.float32, device=dev) if want_d_initial_state else None
    ws, nb = _workspace(dev, "gdn_ssm_bwd_workspace_bytes", sh, workspace)
    _call(dev, "gdn_ssm_bwd", _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(initial_state), _p(cu), _p(dy),
          _p(d_final_state), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC), _p(dD), _p(dbias), _p(dh), ctypes.byref(sh), _p(ws),
          nb)
    return dx, ddt, dA, dB, dC, dD, dbias, dh


def check_ssm_step_args(x, dt, A, B, C, state, D=None, dt_bias=None, slots=None, state_out=None, dt_softplus=True,
                        require_cuda=True):
    """Checks ssm_step's arguments; returns the GdnSsmShape."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or x.numel() < 1:
        _fail("x must be a 3-D tensor [R, H, p] with R, H >= 1")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        _fail("B must be a 3-D tensor [R, G, n]")
    R, H, p = x.shape
    G, n = B.shape[1:]
    dev = x.device
    if G < 1 or H % G:
        _fail("the groups of B (%d) must divide the heads of x (%d)" % (G, H))
    if n not in (64, 128) or p not in (64, 128):
        _fail("state size %d and head size %d must be 64 or 128" % (n, p))
    _check(x, "x", _FP, (R, H, p), dev, require_cuda)
    _check(B, "B", (x.dtype,), (R, G, n), dev, require_cuda)
    _check(C, "C", (x.dtype,), (R, G, n), dev, require_cuda)
    _check(dt, "dt", _FP, (R, H), dev, require_cuda, 1)
    _check_params(A, D, dt_bias, H, dev, require_cuda)
    S = _check_slots(state, state_out, slots, R, (H, n, p), torch.float32, dev, require_cuda)
    return GdnSsmShape(R, 1, H, G, n, p, S, 0, 0, 0, _TYPES[x.dtype], _TYPES[dt.dtype], _TYPES[A.dtype],
                       int(bool(dt_softplus)), 0, 0, None)


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, slots=None, state_out=None, dt_softplus=True, out=None):
    """ssm_fwd for one token of each of R rows: x [R, H, p], dt [R, H], B, C [R, G, n], state
    [S, H, n, p] fp32.  Returns y; slots and state_out as in conv_step."""
    sh = check_ssm_step_args(x, dt, A, B, C, state, D, dt_bias, slots, state_out, dt_softplus)
    _check_out(out, "out", x.dtype, x.shape, x.device, True, (x, dt, A, B, C, D, dt_bias, state, state_out))
    y = out if out is not None else torch.empty_like(x)
    _call(x.device, "gdn_ssm_step", _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias), _p(state), _p(slots), _p(y),
          _p(state if state_out is None else state_out), ctypes.byref(sh))
    return y


# ---- the gated delta rule's step ------------------------------------------------------

def check_delta_step_args(q, k, v, g, beta, state, slots=None, state_out=None, scale=None, require_cuda=True):
    """Checks delta_step's arguments; returns the GdnShape."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.numel() < 1 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        _fail("q must be a 3-D tensor [R, H, dk] with R, H >= 1, v one [R, H, dv]")
    if scale is not None and not math.isfinite(ctypes.c_float(scale).value):
        _fail("scale must be a finite fp32 number")
    R, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    if dk not in (64, 128) or dv not in (64, 128):
        _fail("dk %d and dv %d must be 64 or 128" % (dk, dv))
    _check(q, "q", _FP, (R, H, dk), dev, require_cuda)
    _check(k, "k", (q.dtype,), (R, H, dk), dev, require_cuda)
    _check(v, "v", (q.dtype,), (R, H, dv), dev, require_cuda)
    _check(g, "g", _F32, (R, H), dev, require_cuda, 1)
    _check(beta, "beta", _FP, (R, H), dev, require_cuda, 1)
    S = _check_slots(state, state_out, slots, R, (H, dk, dv), torch.float32, dev, require_cuda)
    return GdnShape(R, 1, H, dk, dv, S, _TYPES[q.dtype], _TYPES[beta.dtype], None)


def delta_step(q, k, v, g, beta, state, scale=None, slots=None, state_out=None, out=None):
    """One token of the gated delta rule for each of R rows (binding.chunk_fwd with T = 1):
    q, k [R, H, dk], v [R, H, dv], g fp32 and beta [R, H], state [S, H, dk, dv] fp32.  Returns o
    [R, H, dv]; slots and state_out as in conv_step."""
    sh = check_delta_step_args(q, k, v, g, beta, state, slots, state_out, scale)
    _check_out(out, "out", q.dtype, v.shape, q.device, True, (q, k, v, g, beta, state, state_out))
    o = out if out is not None else torch.empty_like(v)
    _call(q.device, "gdn_delta_step", _p(q), _p(k), _p(v), _p(g), _p(beta), _p(state), _p(slots),
          1.0 / math.sqrt(sh.dk) if scale is None else scale, _p(o), _p(state if state_out is None else state_out),
          ctypes.byref(sh))
    return o


# ---- norm of the heads' outputs -------------------------------------------------------

def check_norm_args(x, weight=None, bias=None, gate=None, eps=1e-5, require_cuda=True):
    """Checks the norm's inputs; returns (GdnNormShape, shape of the statistics)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        _fail("x must be a tensor [..., D] or [..., H, D]")
    par = weight if weight is not None else bias
    if par is not None and (not isinstance(par, torch.Tensor) or par.dim() not in (1, 2)):
        _fail("weight and bias must be tensors [D] or [H, D]")
    D = x.shape[-1]
    H = par.shape[0] if par is not None and par.dim() == 2 else 1
    if D < 1 or H < 1 or x.numel() == 0 and x.shape[-1] == 0:
        _fail("rows must not be empty")
    if par is not None and par.dim() == 2 and x.shape[-2] != H:
        _fail("x has %d heads, weight and bias have %d" % (x.shape[-2], H))
    if D > 8192:
        _fail("rows of %d elements: at most 8192" % D)
    _check(x, "x", _FP, x.shape, x.device, require_cuda)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check(t, name, (par.dtype,) if par.dtype in _FP else _FP, (H, D) if par.dim() == 2 else (D,), x.device,
                   require_cuda)
    if gate is not None:
        _check(gate, "gate", (x.dtype,), x.shape, x.device, require_cuda)
    if not 0 < ctypes.c_float(eps).value < math.inf:
        _fail("eps must be a positive fp32 number")
    return GdnNormShape(x.numel() // (H * D), H, D, _TYPES[x.dtype], _TYPES[x.dtype if par is None else par.dtype], eps,
                        0), x.shape[:-1]


def norm_fwd(x, weight=None, bias=None, gate=None, eps=1e-5, output_stats=True, out=None):
    """Layer norm over the last axis of x, with a weight and bias [D], or [H, D] for x [..., H, D]
    (each head its own), times silu(gate) if a gate of x's shape is given:

        y = ((x - mean) rstd weight + bias) silu(gate),   rstd = (var + eps)^-1/2

    Returns ``(y, mean, rstd)``, the statistics fp32 (None unless wanted) for norm_bwd."""
    sh, stats = check_norm_args(x, weight, bias, gate, eps)
    _check_out(out, "out", x.dtype, x.shape, x.device, True, (x, weight, bias, gate))
    y = out if out is not None else torch.empty_like(x)
    mean, rstd = (torch.empty(stats, dtype=torch.float32, device=x.device) if output_stats else None for _ in range(2))
    _call(x.device, "gdn_norm_fwd", _p(x), _p(weight), _p(bias), _p(gate), _p(y), _p(mean), _p(rstd), ctypes.byref(sh))
    return y, mean, rstd


def norm_bwd(x, mean, rstd, dy, weight=None, bias=None, gate=None, workspace=None):
    """Gradients of <dy, y> of norm_fwd, from the statistics it returned.  Returns ``(dx,
    dweight, dbias, dgate)`` in the types of what they belong to (None for what is not
    there)."""
    sh, stats = check_norm_args(x, weight, bias, gate)
    _check(dy, "dy", (x.dtype,), x.shape, x.device, True)
    _check(mean, "mean", _F32, stats, x.device, True, 1)
    _check(rstd, "rstd", _F32, stats, x.device, True, 1)
    dx = torch.empty_like(x)
    dw, db, dz = (None if t is None else torch.empty_like(t) for t in (weight, bias, gate))
    ws, nb = None, 0
    if dw is not None or db is not None:
        ws, nb = _workspace(x.device, "gdn_norm_bwd_workspace_bytes", sh, workspace)
    _call(x.device, "gdn_norm_bwd", _p(x), _p(weight), _p(bias), _p(gate), _p(mean), _p(rstd), _p(dy), _p(dx), _p(dw),
          _p(db), _p(dz), ctypes.byref(sh), _p(ws), nb)
    return dx, dw, db, dz
