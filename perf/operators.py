"""What the token mixers' operators beside the chunked gated delta rule are measured on: the short causal
convolution, the selective state space scan, the norm of the heads' outputs and the single-token steps.

``run`` computes them in plain form (elementary torch operations in 32 bits, log decays and long sums in 64), or, where
``own`` is true, makes the calls a user makes of ``gated_deltanet_chunked_fwd_amd.mixer``.  ``exact`` computes
the same outputs from the definitions, token by token, in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # convolution of the concatenated q, k, v channels (16 heads of 128, three times) of a prompt batch
        dict(name="conv_prompt", op="conv_fwd", B=4, T=4096, D=6144, W=4, dtype="bf16", lens="", state=False, bias=False),
        # its gradients in a training step on packed documents, one of them shorter than the taps
        dict(name="conv_train_packed", op="conv_bwd", B=1, T=12003, D=2312, W=4, dtype="bf16",
             lens="2,4093,1,0,3000,4907", state=True, bias=True),
        # one new token for each of 64 sequences, states in a pool of slots
        dict(name="conv_decode", op="conv_step", R=64, S=96, D=6144, W=4, dtype="bf16", bias=True),
        # the scan over a prompt batch, B and C shared by all heads
        dict(name="scan_prompt", op="ssm_fwd", B=4, T=4096, H=16, G=1, n=128, p=128, dtype="bf16", params="f32",
             lens="", state=False),
        # one long document on few heads, each with its own B and C: the sequence has to be split
        dict(name="scan_long", op="ssm_fwd", B=1, T=131072, H=4, G=4, n=128, p=128, dtype="bf16", params="f32",
             lens="", state=True),
        # gradients of a training step on packed documents, two groups of heads
        dict(name="scan_train_packed", op="ssm_bwd", B=1, T=8192, H=16, G=2, n=128, p=64, dtype="bf16", params="bf16",
             lens="1700,64,0,3333,1,3094", state=True),
        # gradients in 32 bits, as a numerics check of a small model runs them
        dict(name="scan_train_f32", op="ssm_bwd", B=2, T=777, H=4, G=4, n=64, p=64, dtype="f32", params="f32",
             lens="", state=False),
        # one new token for each of 64 sequences
        dict(name="scan_decode", op="ssm_step", R=64, S=80, H=16, G=1, n=128, p=128, dtype="bf16", params="f32"),
        # each head's output normalised and gated, on the prompt batch
        dict(name="norm_heads_gated", op="norm_fwd", rows=16384, H=16, D=128, dtype="bf16", affine=True, gate=True),
        # gradients of the residual stream's norm (one head as wide as the model) in a training step
        dict(name="norm_train", op="norm_bwd", rows=16384, H=1, D=2048, dtype="bf16", affine=True, gate=False),
        # the gated delta rule's next token of a single sequence: latency alone counts
        dict(name="delta_decode_one", op="delta_step", R=1, S=1, H=16, dk=128, dv=128, dtype="bf16"),
        # and of a full batch
        dict(name="delta_decode_batch", op="delta_step", R=256, S=256, H=16, dk=128, dv=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, T):
    """A text of packed lengths that sum to T, empty ones among them."""
    cuts = sorted(rng.randrange(T + 1) for _ in range(rng.randrange(1, 9)))
    edges = [0] + cuts + [T]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_bwd", "ssm_step",
                     "norm_fwd", "norm_bwd", "delta_step"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op in ("conv_fwd", "conv_bwd"):
        D = _log(rng, 64, 8192)
        tokens = _log(rng, 1, min(100000, (60_000_000 if dtype == "bf16" else 25_000_000) // D))
        packed = rng.random() < 0.4
        B = 1 if packed else rng.choice([1, 1, 2, 3])
        T = max(1, tokens // B)
        return dict(op=op, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), dtype=dtype, lens=_lens(rng, T) if packed else "",
                    state=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op == "conv_step":
        R = _log(rng, 1, 512)
        return dict(op=op, R=R, S=R + rng.randrange(40), D=_log(rng, 64, 8192), W=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    bias=rng.random() < 0.5)
    if op in ("ssm_fwd", "ssm_bwd"):
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4, 8])
        n, p = rng.choice([64, 128]), rng.choice([64, 128])
        packed = rng.random() < 0.4
        B = 1 if packed else rng.choice([1, 1, 2, 3])
        T = max(1, _log(rng, 1, (400_000 if op == "ssm_fwd" else 120_000) // H) // B)
        if dtype == "f32":
            T = min(T, 4000)
        return dict(op=op, B=B, T=T, H=H, G=G, n=n, p=p, dtype=dtype, params=dtype if op == "ssm_bwd" else "f32",
                    lens=_lens(rng, T) if packed else "", state=rng.random() < 0.5)
    if op == "ssm_step":
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4, 8])
        R = _log(rng, 1, min(256, 3200 // H))
        return dict(op=op, R=R, S=R + rng.randrange(20), H=H, G=G, n=rng.choice([64, 128]),
                    p=rng.choice([64, 128]), dtype=dtype, params="f32")
    if op in ("norm_fwd", "norm_bwd"):
        H = rng.choice([1, 1, 4, 5, 16, 32])
        D = rng.choice([64, 96, 128, 256]) if H > 1 else _log(rng, 64, 8192)
        return dict(op=op, rows=_log(rng, 1, min(50000, 25_000_000 // (H * D))), H=H, D=D, dtype=dtype,
                    affine=rng.random() < 0.8, gate=rng.random() < 0.5)
    R = _log(rng, 1, 256)
    return dict(op=op, R=R, S=R + rng.randrange(20), H=rng.choice([1, 2, 4, 5, 8, 12]), dk=rng.choice([64, 128]),
                dv=rng.choice([64, 128]), dtype=dtype)


# ---- inputs -------------------------------------------------------------------------------------------------

def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return (lambda *s: torch.randn(s, generator=g, device="cuda"), lambda *s: torch.rand(s, generator=g, device="cuda"),
            lambda n: torch.randperm(n, generator=g, device="cuda"))


def _sequences(case):
    """(lengths, device cu_seqlens, host cu_seqlens); the last two None where sequences are batch rows."""
    if not case["lens"]:
        return [case["T"]] * case["B"], None, None
    lens = [int(v) for v in case["lens"].split(",")]
    host = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    return lens, host.cuda(), host


def prepare(case, seed):
    randn, rand, perm = _maker(seed)
    e, op = TYPES[case["dtype"]], case["op"]
    s = dict(case=case)
    if op in ("conv_fwd", "conv_bwd"):
        B, T, D, W = case["B"], case["T"], case["D"], case["W"]
        s["lens"], s["cu"], s["host"] = _sequences(case)
        N = len(s["lens"])
        s["x"] = randn(B, T, D).to(e)
        s["weight"] = (randn(D, W) * W ** -0.5).to(e)
        s["bias"] = (randn(D) * 0.1).to(e) if case["bias"] else None
        s["init"] = randn(N, W - 1, D).to(e) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = randn(B, T, D).to(e)
            s["dfin"] = randn(N, W - 1, D).to(e) if case["state"] else None
    elif op == "conv_step":
        R, S, D, W = case["R"], case["S"], case["D"], case["W"]
        s.update(x=randn(R, D).to(e), weight=(randn(D, W) * W ** -0.5).to(e), state=randn(S, W - 1, D).to(e),
                 bias=(randn(D) * 0.1).to(e) if case["bias"] else None, slots=perm(S)[:R].to(torch.int32))
        s["state_out"] = torch.zeros_like(s["state"])
    elif op in ("ssm_fwd", "ssm_bwd", "ssm_step"):
        H, G, n, p, pe = case["H"], case["G"], case["n"], case["p"], TYPES[case["params"]]
        step = op == "ssm_step"
        lead = (case["R"],) if step else (case["B"], case["T"])
        s["x"] = torch.nn.functional.silu(randn(*lead, H, p)).to(e)
        s["dt"] = (randn(*lead, H) * 0.5).to(e)
        s["b"] = torch.nn.functional.silu(randn(*lead, G, n)).to(e)
        s["c"] = torch.nn.functional.silu(randn(*lead, G, n)).to(e)
        s["A"] = (-(1.0 + 15.0 * rand(H))).to(pe)
        s["D"] = (1.0 + 0.1 * randn(H)).to(pe)
        dt0 = torch.exp(rand(H) * math.log(100.0) + math.log(0.001))   # softplus(dt_bias) from 0.001 to 0.1
        s["dt_bias"] = torch.log(torch.expm1(dt0)).to(pe)
        if step:
            S = case["S"]
            s.update(state=randn(S, H, n, p) * 0.3, slots=perm(S)[:case["R"]].to(torch.int32))
            s["state_out"] = torch.zeros_like(s["state"])
            return s
        s["lens"], s["cu"], s["host"] = _sequences(case)
        N = len(s["lens"])
        s["h0"] = randn(N, H, n, p) * 0.3 if case["state"] else None
        if op == "ssm_bwd":
            s["dy"] = randn(*lead, H, p).to(e)
            s["dhT"] = randn(N, H, n, p) * 0.3 if case["state"] else None
    elif op in ("norm_fwd", "norm_bwd"):
        rows, H, D = case["rows"], case["H"], case["D"]
        s["x"] = (randn(rows, H, D) * 1.5 + 0.5 * randn(rows, H, 1)).to(e)
        s["weight"] = (1.0 + 0.1 * randn(H, D)).to(e) if case["affine"] else None
        s["bias"] = (0.1 * randn(H, D)).to(e) if case["affine"] else None
        s["gate"] = randn(rows, H, D).to(e) if case["gate"] else None
        if op == "norm_bwd":   # the statistics that the forward pass kept
            s["dy"] = randn(rows, H, D).to(e)
            x = s["x"].double()
            s["mean"] = x.mean(-1).float()
            s["rstd"] = torch.rsqrt(x.var(-1, unbiased=False) + 1e-5).float()
    else:
        R, S, H, dk, dv = case["R"], case["S"], case["H"], case["dk"], case["dv"]
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
        s.update(q=unit(randn(R, H, dk)).to(e), k=unit(randn(R, H, dk)).to(e), v=randn(R, H, dv).to(e),
                 g=torch.nn.functional.logsigmoid(randn(R, H) + 3.0), beta=torch.sigmoid(randn(R, H)).to(e),
                 state=randn(S, H, dk, dv) * 0.3, slots=perm(S)[:R].to(torch.int32))
        s["state_out"] = torch.zeros_like(s["state"])
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------

def _f(t):
    return None if t is None else t.float()


def _to_rows(s, t):
    """Packed tokens [1, T, ...] as [N, longest, ...], zeros behind each sequence; batch rows as they are."""
    if s["cu"] is None:
        return t
    cu, N, L = s["cu"].long(), len(s["lens"]), max(s["lens"])
    at = cu[:-1, None] + torch.arange(L, device=t.device)
    real = at < cu[1:, None]
    return t[0][at.clamp(max=t.shape[1] - 1)] * real.reshape(N, L, *[1] * (t.dim() - 2)).to(t.dtype)


def _to_tokens(s, t):
    """The real tokens of [N, longest, ...], packed again."""
    if s["cu"] is None:
        return t
    cu, L = s["cu"].long(), t.shape[1]
    at = torch.arange(L, device=t.device)
    return t[at < (cu[1:, None] - cu[:-1, None])][None]


def _lengths(s, like):
    return torch.tensor(s["lens"], device=like.device)


def _conv_parts(s):
    """(inputs with the state in front, their windows [N, L, D, W], z)."""
    c = s["case"]
    x = _to_rows(s, _f(s["x"]))
    first = _f(s["init"]) if s["init"] is not None else x.new_zeros(x.shape[0], c["W"] - 1, c["D"])
    xe = torch.cat([first, x], 1)
    win = xe.unfold(1, c["W"], 1)
    z = (win * _f(s["weight"])).sum(-1)
    return xe, win, z if s["bias"] is None else z + _f(s["bias"])


def _plain_conv_fwd(s):
    e, W = s["x"].dtype, s["case"]["W"]
    xe, _, z = _conv_parts(s)
    last = _lengths(s, xe)[:, None] + torch.arange(W - 1, device=xe.device)
    fin = xe.gather(1, last[..., None].expand(-1, -1, xe.shape[2]))
    return _to_tokens(s, z * torch.sigmoid(z)).to(e), fin.to(e)


def _plain_conv_bwd(s):
    e, W = s["x"].dtype, s["case"]["W"]
    xe, win, z = _conv_parts(s)
    sg = torch.sigmoid(z)
    dz = _to_rows(s, _f(s["dy"])) * (sg * (1 + z * (1 - sg)))
    dw = (win * dz[..., None]).sum((0, 1))
    dxe = (torch.nn.functional.pad(dz, (0, 0, W - 1, W - 1)).unfold(1, W, 1) * _f(s["weight"]).flip(-1)).sum(-1)
    if s["dfin"] is not None:
        last = _lengths(s, xe)[:, None] + torch.arange(W - 1, device=xe.device)
        dxe = dxe.scatter_add(1, last[..., None].expand(-1, -1, xe.shape[2]), _f(s["dfin"]))
    return (_to_tokens(s, dxe[:, W - 1:]).to(e), dw.to(e), None if s["bias"] is None else dz.sum((0, 1)).to(e),
            None if s["init"] is None else dxe[:, :W - 1].to(e))


def _plain_conv_step(s):
    e, at = s["x"].dtype, s["slots"].long()
    win = torch.cat([s["state"][at], s["x"][:, None]], 1)
    z = (win.float() * _f(s["weight"]).t()).sum(1)
    z = z if s["bias"] is None else z + _f(s["bias"])
    s["state_out"].index_copy_(0, at, win[:, 1:])
    return (z * torch.sigmoid(z)).to(e), s["state_out"]


def _scan(q, k, v, a, h0):
    """out_t = q_t h_t, h_t = exp(a_t) h_{t-1} + k_t v_t^T, in chunks; a in 64 bits.  Returns out and the last h."""
    N, L, H, _ = q.shape
    pad = -L % CHUNK
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, pad)) for t in (q, k, v))
    a = torch.nn.functional.pad(a, (0, 0, 0, pad))
    nc = (L + pad) // CHUNK
    q, k, v = (t.reshape(N, nc, CHUNK, H, -1).transpose(2, 3).contiguous() for t in (q, k, v))
    G = a.reshape(N, nc, CHUNK, H).transpose(2, 3).cumsum(-1)                       # [N, nc, H, CHUNK]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).to(q.dtype)
    out = ((q @ k.transpose(-1, -2).contiguous()) * decay) @ v
    end = G[..., -1:]
    S = (k * torch.exp(end - G).to(q.dtype)[..., None]).transpose(-1, -2).contiguous() @ v   # [N, nc, H, dk, dv]
    first = torch.zeros_like(S[:, :1]) if h0 is None else h0[:, None]
    S = torch.cat([first, S], 1)                                                    # what enters at each chunk's end
    cum = torch.nn.functional.pad(end[..., 0].cumsum(1), (0, 0, 1, 0)).transpose(1, 2)     # [N, H, nc + 1]
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=q.device).tril()
    carry = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf)).to(q.dtype)
    h = carry @ S.transpose(1, 2).reshape(N, H, nc + 1, -1)
    h = h.reshape(N, H, nc + 1, *S.shape[-2:]).transpose(1, 2)
    out = out + (q * torch.exp(G).to(q.dtype)[..., None]) @ h[:, :-1].contiguous()
    return out.transpose(2, 3).reshape(N, L + pad, H, -1)[:, :L], h[:, -1]


def _rev_scan(q, k, v, a, hT):
    """out_s = q_s g_s, g_s = exp(a_{s+1}) g_{s+1} + k_s v_s^T, hT behind the last.  Returns out and exp(a_0) g_0."""
    a1 = torch.nn.functional.pad(a[:, 1:], (0, 0, 0, 1))
    out, g = _scan(q.flip(1), k.flip(1), v.flip(1), a1.flip(1), hT)
    return out.flip(1), g * torch.exp(a[:, 0]).to(g.dtype)[..., None, None]


def _ssm_parts(s, wide=torch.float32):
    c = s["case"]
    r = c["H"] // c["G"]
    x, dt, b, cc = (_to_rows(s, s[k].to(wide)) for k in ("x", "dt", "b", "c"))
    delta = torch.nn.functional.softplus(dt + s["dt_bias"].to(wide))
    if s["cu"] is not None:   # nothing happens behind a sequence's end
        delta = delta * (torch.arange(x.shape[1], device=x.device) < _lengths(s, x)[:, None])[..., None]
    a = delta.double() * s["A"].double()
    return x, dt, delta, a, b.repeat_interleave(r, 2), cc.repeat_interleave(r, 2)


def _plain_ssm_fwd(s):
    x, dt, delta, a, b, c = _ssm_parts(s)
    y, hT = _scan(c, b * delta[..., None], x, a, s["h0"])
    return _to_tokens(s, y + x * _f(s["D"])[:, None]).to(s["x"].dtype), hT


def _plain_ssm_bwd(s):
    # the parameters' gradients are long sums of flows that nearly cancel: 32 bits hold 32-bit ones to 2e-5 only
    case, e, pe = s["case"], s["x"].dtype, s["A"].dtype
    wide = torch.float64 if pe == torch.float32 else torch.float32
    x, dt, delta, a, b, c = _ssm_parts(s, wide)
    dy = _to_rows(s, s["dy"].to(wide))
    dl = delta[..., None]
    h0, dhT = (None if s[k] is None else s[k].to(wide) for k in ("h0", "dhT"))
    turn = lambda h: None if h is None else h.transpose(-1, -2).contiguous()  # noqa: E731
    dC, hT = _scan(dy, x * dl, b, a, turn(h0))
    dB, _ = _rev_scan(x, dy, c, a, turn(dhT))
    dB = dB * dl
    du, dh0 = _rev_scan(b, c, dy, a, dhT)
    flow = (c.double() * dC.double()).sum(-1) - (b.double() * dB.double()).sum(-1)
    da = flow.flip(1).cumsum(1).flip(1)
    if dhT is not None:
        da = da + (hT.double() * turn(dhT).double()).sum((-1, -2))[:, None]
    ddelta = (x * du).sum(-1).double() + da * s["A"].double()
    ddt = ddelta * torch.sigmoid(dt.double() + s["dt_bias"].double())
    ddt = _to_tokens(s, ddt)
    groups = lambda t: _to_tokens(s, t.reshape(*t.shape[:2], case["G"], -1, case["n"]).sum(3)).to(e)  # noqa: E731
    dx = du * dl + dy * s["D"].to(wide)[:, None]
    dA = (_to_tokens(s, delta).double() * _to_tokens(s, da)).sum((0, 1))
    return (_to_tokens(s, dx).to(e), ddt.to(e), dA.to(pe), groups(dB), groups(dC),
            (dy.double() * x.double()).sum((0, 1, 3)).to(pe), ddt.sum((0, 1)).to(pe), None if h0 is None else dh0.float())


def _plain_ssm_step(s):
    c, at = s["case"], s["slots"].long()
    r = c["H"] // c["G"]
    x, delta = _f(s["x"]), torch.nn.functional.softplus(_f(s["dt"]) + _f(s["dt_bias"]))
    b, cc = (_f(s[k]).repeat_interleave(r, 1) for k in ("b", "c"))
    h = s["state"][at] * torch.exp(delta * _f(s["A"]))[..., None, None]
    h = h + (b * delta[..., None])[..., :, None] * x[..., None, :]
    s["state_out"].index_copy_(0, at, h)
    return ((cc[..., :, None] * h).sum(-2) + x * _f(s["D"])[:, None]).to(s["x"].dtype), s["state_out"]


def _plain_norm_fwd(s):
    x = _f(s["x"])
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + 1e-5)
    y = (x - mean) * rstd
    if s["weight"] is not None:
        y = y * _f(s["weight"]) + _f(s["bias"])
    if s["gate"] is not None:
        z = _f(s["gate"])
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype), mean[..., 0], rstd[..., 0]


def _plain_norm_bwd(s):
    e = s["x"].dtype
    dy, rstd = _f(s["dy"]), s["rstd"][..., None]
    xh = (_f(s["x"]) - s["mean"][..., None]) * rstd
    w = 1.0 if s["weight"] is None else _f(s["weight"])
    dz = None
    if s["gate"] is not None:
        z = _f(s["gate"])
        sg = torch.sigmoid(z)
        dz = (dy * (xh * w + (0.0 if s["bias"] is None else _f(s["bias"]))) * (sg * (1 + z * (1 - sg)))).to(e)
        dy = dy * (z * sg)
    dw = None if s["weight"] is None else (dy * xh).sum(0).to(e)
    db = None if s["bias"] is None else dy.sum(0).to(e)
    dxh = dy * w
    dx = rstd * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    return dx.to(e), dw, db, dz


def _plain_delta_step(s):
    at = s["slots"].long()
    q, k, v, beta = _f(s["q"]), _f(s["k"]), _f(s["v"]), _f(s["beta"])
    h = s["state"][at] * torch.exp(s["g"])[..., None, None]
    u = beta[..., None] * (v - (k[..., :, None] * h).sum(-2))
    h = h + k[..., :, None] * u[..., None, :]
    s["state_out"].index_copy_(0, at, h)
    return ((q[..., :, None] * h).sum(-2) * q.shape[-1] ** -0.5).to(s["q"].dtype), s["state_out"]


PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
         "ssm_fwd": _plain_ssm_fwd, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step,
         "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "delta_step": _plain_delta_step}


# ---- the framework's calls ----------------------------------------------------------------------------------

def _own(s):
    from gated_deltanet_chunked_fwd_amd import mixer
    op = s["case"]["op"]
    if op == "conv_fwd":
        return mixer.conv_fwd(s["x"], s["weight"], s["bias"], initial_state=s["init"], cu_seqlens=s["cu"],
                              cu_seqlens_host=s["host"])
    if op == "conv_bwd":
        return mixer.conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], initial_state=s["init"], d_final_state=s["dfin"],
                              cu_seqlens=s["cu"], cu_seqlens_host=s["host"], want_d_initial_state=s["init"] is not None)
    if op == "conv_step":
        return mixer.conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"], state_out=s["state_out"]), s["state_out"]
    if op == "ssm_fwd":
        return mixer.ssm_fwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"], initial_state=s["h0"],
                             cu_seqlens=s["cu"], cu_seqlens_host=s["host"])
    if op == "ssm_bwd":
        return mixer.ssm_bwd(s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"], s["dy"], initial_state=s["h0"],
                             d_final_state=s["dhT"], cu_seqlens=s["cu"], cu_seqlens_host=s["host"],
                             want_d_initial_state=s["h0"] is not None)
    if op == "ssm_step":
        return mixer.ssm_step(s["x"], s["dt"], s["A"], s["b"], s["c"], s["state"], s["D"], s["dt_bias"], slots=s["slots"],
                              state_out=s["state_out"]), s["state_out"]
    if op == "norm_fwd":
        return mixer.norm_fwd(s["x"], s["weight"], s["bias"], gate=s["gate"])
    if op == "norm_bwd":
        return mixer.norm_bwd(s["x"], s["mean"], s["rstd"], s["dy"], s["weight"], s["bias"], gate=s["gate"])
    return mixer.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"],
                            state_out=s["state_out"]), s["state_out"]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("conv_fwd", "conv_bwd"):
        n = case["B"] * case["T"] * case["D"]
        N = len(case["lens"].split(",")) if case["lens"] else case["B"]
        st = N * (case["W"] - 1) * case["D"] * e
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + st * (1 + case["state"]), "flops": 2 * n * case["W"]}
        return {"bytes": 3 * n * e + 3 * st * case["state"] + 2 * case["D"] * case["W"] * e, "flops": 6 * n * case["W"]}
    if op == "conv_step":
        n = case["R"] * case["D"]
        return {"bytes": (2 * n + 2 * n * (case["W"] - 1) + case["D"] * case["W"]) * e, "flops": 2 * n * case["W"]}
    if op in ("norm_fwd", "norm_bwd"):
        n = case["rows"] * case["H"] * case["D"]
        k = (2 if op == "norm_fwd" else 3) + case["gate"] * (1 if op == "norm_fwd" else 2)
        return {"bytes": k * n * e + 8 * case["rows"] * case["H"], "flops": 12 * n}
    if op == "delta_step":
        n = case["R"] * case["H"]
        return {"bytes": n * (8 * case["dk"] * case["dv"] + (2 * case["dk"] + 2 * case["dv"]) * e), "flops": 7 * n * case["dk"] * case["dv"]}
    H, G, n, p = case["H"], case["G"], case["n"], case["p"]
    if op == "ssm_step":
        R = case["R"]
        return {"bytes": R * H * (8 * n * p + 2 * p * e) + 2 * R * G * n * e, "flops": 5 * R * H * n * p}
    tokens = case["B"] * case["T"]
    N = len(case["lens"].split(",")) if case["lens"] else case["B"]
    io = tokens * (H * p + 2 * G * n + H) * e   # x, B, C and dt, or as many gradients
    states = N * H * n * p * 4
    scan = tokens * H * (CHUNK * (n + p) + 4 * n * p)   # the triangle inside a chunk, and the state read and updated
    if op == "ssm_fwd":
        return {"bytes": io + tokens * H * p * e + states * (1 + case["state"]), "flops": scan}
    # dy beside x, B, C, dt; their gradients; h_0, dh_T and dh_0.  Both states are built again, each read by two products.
    return {"bytes": 2 * io + tokens * H * p * e + 3 * states * case["state"],
            "flops": tokens * H * (CHUNK * (n + p) + CHUNK * (2 * n + p) + 10 * n * p)}


# ---- in 64 bits, from the definitions -----------------------------------------------------------------------

def _pieces(s):
    """(batch row, first token, end) of each sequence."""
    if s["cu"] is None:
        return [(i, 0, n) for i, n in enumerate(s["lens"])]
    ends = [int(v) for v in s["host"]]
    return [(0, a, b) for a, b in zip(ends, ends[1:])]


def _exact_conv(s, case):
    W, D, back = case["W"], case["D"], case["op"] == "conv_bwd"
    x, w = s["x"].double(), s["weight"].double()
    bias = torch.zeros(D, dtype=torch.float64, device=x.device) if s["bias"] is None else s["bias"].double()
    ys, fins, dws, inits = torch.zeros_like(x), [], torch.zeros_like(w), []
    dbias = torch.zeros_like(bias)
    for i, (row, a, b) in enumerate(_pieces(s)):
        old = x.new_zeros(W - 1, D) if s["init"] is None else s["init"][i].double()
        full = torch.cat([old, x[row, a:b]])
        n = b - a
        z = bias.expand(n, D).clone()
        for j in range(W):
            z += w[:, j] * full[j:j + n]
        gate = 1 / (1 + torch.exp(-z))
        if not back:
            ys[row, a:b] = z * gate
            fins.append(full[n:])
            continue
        dz = s["dy"][row, a:b].double() * (gate + z * gate * (1 - gate))
        dfull = torch.zeros_like(full)
        for j in range(W):
            dfull[j:j + n] += w[:, j] * dz
            dws[:, j] += (dz * full[j:j + n]).sum(0)
        if s["dfin"] is not None:
            dfull[n:] += s["dfin"][i].double()
        ys[row, a:b] = dfull[W - 1:]
        inits.append(dfull[:W - 1])
        dbias += dz.sum(0)
    if not back:
        return ys, torch.stack(fins)
    return ys, dws, None if s["bias"] is None else dbias, None if s["init"] is None else torch.stack(inits)


def _exact_ssm(s, case):
    back = case["op"] == "ssm_bwd"
    H, G, n, p = case["H"], case["G"], case["n"], case["p"]
    x, A, D = s["x"].double(), s["A"].double(), s["D"].double()
    raw = s["dt"].double() + s["dt_bias"].double()
    delta = torch.log1p(torch.exp(raw))
    b, c = s["b"].double(), s["c"].double()
    head = torch.arange(H, device=x.device) // (H // G)
    y, ends = torch.zeros_like(x), []
    dx, ddelta, da_sum = torch.zeros_like(x), torch.zeros_like(delta), torch.zeros_like(A)
    db, dc, starts = torch.zeros_like(b), torch.zeros_like(c), []
    fold = lambda t: t.reshape(G, H // G, -1).sum(1)  # noqa: E731
    for i, (row, t0, t1) in enumerate(_pieces(s)):
        h = x.new_zeros(H, n, p) if s["h0"] is None else s["h0"][i].double()
        if not back:
            for t in range(t0, t1):
                d = delta[row, t]
                h = h * torch.exp(d * A)[:, None, None] + (b[row, t][head] * d[:, None])[:, :, None] * x[row, t][:, None, :]
                y[row, t] = (c[row, t][head][:, :, None] * h).sum(1)
            ends.append(h)
            continue
        step, kept = 128, []          # states kept every 128 tokens, the ones between built again on the way back
        def forward(h, lo, hi, into=None):
            for t in range(lo, hi):
                if into is not None:
                    into.append(h)
                d = delta[row, t]
                h = h * torch.exp(d * A)[:, None, None] + (b[row, t][head] * d[:, None])[:, :, None] * x[row, t][:, None, :]
            return h
        for lo in range(t0, t1, step):
            kept.append((lo, h))
            h = forward(h, lo, min(t1, lo + step))
        dh = torch.zeros_like(h) if s["dhT"] is None else s["dhT"][i].double()
        for lo, h in reversed(kept):
            hs = []
            end = forward(h, lo, min(t1, lo + step), hs)
            for t in range(min(t1, lo + step) - 1, lo - 1, -1):
                d, dy, xt, bt = delta[row, t], s["dy"][row, t].double(), x[row, t], b[row, t][head]
                dh = dh + c[row, t][head][:, :, None] * dy[:, None, :]
                dc[row, t] = fold((end * dy[:, None, :]).sum(2))
                xs = (dh * xt[:, None, :]).sum(2)
                bs = (dh * bt[:, :, None]).sum(1)
                db[row, t] = fold(xs * d[:, None])
                dx[row, t] = bs * d[:, None] + D[:, None] * dy
                keep = torch.exp(d * A)
                da = keep * (hs[t - lo] * dh).sum((1, 2))
                ddelta[row, t] = (bs * xt).sum(1) + A * da
                da_sum += d * da
                dh = dh * keep[:, None, None]
                end = hs[t - lo]
        starts.append(dh)
    if not back:
        return y + x * D[:, None], torch.stack(ends)
    ddt = ddelta / (1 + torch.exp(-raw))
    return (dx, ddt, da_sum, db, dc, (s["dy"].double() * x).sum((0, 1, 3)), ddt.sum((0, 1)),
            None if s["h0"] is None else torch.stack(starts))


def exact(case, seed):
    op = case["op"]
    if op in ("ssm_fwd", "ssm_bwd") and case["B"] * case["T"] > (16384 if op == "ssm_fwd" else 9000):
        return None
    s = prepare(case, seed)
    if op in ("conv_fwd", "conv_bwd"):
        return _exact_conv(s, case)
    if op in ("ssm_fwd", "ssm_bwd"):
        return _exact_ssm(s, case)
    if op in ("norm_fwd", "norm_bwd"):
        x = s["x"].double()
        w = torch.ones_like(x[0]) if s["weight"] is None else s["weight"].double()
        b = torch.zeros_like(x[0]) if s["bias"] is None else s["bias"].double()
        z = None if s["gate"] is None else s["gate"].double()
        if op == "norm_fwd":
            mean, var = x.mean(-1), x.var(-1, unbiased=False)
            rstd = 1 / torch.sqrt(var + 1e-5)
            y = (x - mean[..., None]) * rstd[..., None] * w + b
            return (y if z is None else y * z / (1 + torch.exp(-z))), mean, rstd
        mean, rstd = s["mean"].double()[..., None], s["rstd"].double()[..., None]
        xh, dy, dz = (x - mean) * rstd, s["dy"].double(), None
        if z is not None:
            sg = 1 / (1 + torch.exp(-z))
            dz = dy * (xh * w + b) * (sg + z * sg * (1 - sg))
            dy = dy * z * sg
        gx, D = dy * w, case["D"]
        dx = rstd / D * (D * gx - gx.sum(-1, keepdim=True) - xh * (gx * xh).sum(-1, keepdim=True))
        return (dx, None if s["weight"] is None else (dy * xh).sum(0), None if s["bias"] is None else dy.sum(0), dz)
    slots = [int(v) for v in s["slots"]]
    out = torch.zeros(s["state"].shape, dtype=torch.float64, device="cuda")
    if op == "conv_step":
        ys = []
        for i, j in enumerate(slots):
            win = torch.cat([s["state"][j].double(), s["x"][i:i + 1].double()])
            z = (win * s["weight"].double().t()).sum(0) + (0 if s["bias"] is None else s["bias"].double())
            out[j] = win[1:]
            ys.append(z / (1 + torch.exp(-z)))
        return torch.stack(ys), out
    ys = []
    for i, j in enumerate(slots):
        h = s["state"][j].double()
        if op == "ssm_step":
            head = torch.arange(case["H"], device=h.device) // (case["H"] // case["G"])
            d = torch.log1p(torch.exp(s["dt"][i].double() + s["dt_bias"].double()))
            x = s["x"][i].double()
            h = h * torch.exp(d * s["A"].double())[:, None, None] + (d[:, None] * s["b"][i].double()[head])[:, :, None] * x[:, None, :]
            y = torch.matmul(s["c"][i].double()[head][:, None, :], h)[:, 0] + s["D"].double()[:, None] * x
        else:
            q, k, v = (s[t][i].double() for t in "qkv")
            h = h * torch.exp(s["g"][i].double())[:, None, None]
            u = s["beta"][i].double()[:, None] * (v - torch.matmul(k[:, None, :], h)[:, 0])
            h = h + k[:, :, None] * u[:, None, :]
            y = torch.matmul(q[:, None, :], h)[:, 0] * case["dk"] ** -0.5
        out[j] = h
        ys.append(y)
    return torch.stack(ys), out
