"""Plain 64-bit references of the operators of gated_deltanet_chunked_fwd_amd.mixer: token by
token from their definitions, differentiable (torch autograd gives the gradients), on the
CPU.  Test infrastructure only; nothing here is shared with the library."""
import torch

F64 = torch.float64


def wide(t):
    return None if t is None else t.detach().to("cpu", F64)


def pieces(B, T, lens):
    """(batch row, first token, end) of each sequence."""
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    out, at = [], 0
    for n in lens:
        out.append((0, at, at + n))
        at += n
    assert at == T
    return out


def conv(x, w, bias, init, lens, silu=True):
    B, T, D = x.shape
    W = w.shape[1]
    y, fins = torch.zeros_like(x), []
    for i, (r, a, b) in enumerate(pieces(B, T, lens)):
        old = x.new_zeros(W - 1, D) if init is None else init[i]
        full = torch.cat([old, x[r, a:b]])
        z = sum(full[j:j + b - a] * w[:, j] for j in range(W))
        if bias is not None:
            z = z + bias
        rows = torch.zeros(T, D, dtype=x.dtype)
        rows[a:b] = z * torch.sigmoid(z) if silu else z
        y = y + torch.stack([rows if q == r else torch.zeros_like(rows) for q in range(B)])
        fins.append(full[b - a:])
    return y, torch.stack(fins)


def ssm(x, dt, A, B, C, D, bias, h0, lens, softplus=True):
    """B and C per head: [B, T, H, n]."""
    nb, T, H, p = x.shape
    raw = dt if bias is None else dt + bias
    delta = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    rows = [[None] * T for _ in range(nb)]
    ends = []
    for i, (r, a, b) in enumerate(pieces(nb, T, lens)):
        h = x.new_zeros(H, B.shape[-1], p) if h0 is None else h0[i]
        for t in range(a, b):
            d = delta[r, t]
            h = h * torch.exp(d * A)[:, None, None] + (d[:, None] * B[r, t])[:, :, None] * x[r, t][:, None, :]
            y = (C[r, t][:, :, None] * h).sum(1)
            rows[r][t] = y if D is None else y + D[:, None] * x[r, t]
        ends.append(h)
    y = torch.stack([torch.stack(q) if q else x.new_zeros(0, H, p) for q in rows])
    return y, torch.stack(ends)


def delta_rule(q, k, v, g, beta, h, scale):
    """One token: q, k [H, dk], v [H, dv], g, beta [H], h [H, dk, dv]."""
    h = h * torch.exp(g)[:, None, None]
    u = beta[:, None] * (v - (k[:, :, None] * h).sum(1))
    h = h + k[:, :, None] * u[:, None, :]
    return scale * (q[:, :, None] * h).sum(1), h


def norm(x, w, b, gate, eps):
    """x [..., D]; w, b [D] or [H, D]."""
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    if gate is not None:
        y = y * gate * torch.sigmoid(gate)
    return y, mean[..., 0], rstd[..., 0]
