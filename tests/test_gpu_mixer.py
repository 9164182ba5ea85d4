"""The operators of gated_deltanet_chunked_fwd_amd.mixer on the GPU against 64-bit references
(tests/mixer_ref.py, gradients by autograd).

Tolerances count roundings (u = half a step: bf16 2^-8, fp32 2^-24; all relative).
  * A result in bf16 is rounded once: |err| <= 2^-8 |ref|, plus what its sum is off by.
  * Sums are fp32.  A sum of m products is off by at most m 2^-24 of the sum of the
    products' sizes, which `slack` bounds: the reference computed from absolute values.
  * The scan's bf16 path rounds the state once to bf16 in the forward pass's outputs (2^-8 of
    each product's size), and carries computed operands as two bf16 terms in the backward pass
    (2^-16) and as three in the state's update (2^-24).
"""
import pytest
import torch

from gated_deltanet_chunked_fwd_amd import binding, mixer
from tests import mixer_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
DEV = "cuda"


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g)


def close(got, ref, slack, rel, what):
    """|got - ref| <= u |ref| + rel slack, elementwise (u by got's type)."""
    assert got.shape == ref.shape, what
    got64 = got.detach().cpu().double()
    assert torch.isfinite(got64).all(), what
    off = (got64 - ref).abs()
    tol = U[got.dtype] * ref.abs() + rel * slack + 1e-30
    worst = float((off / tol).max()) if off.numel() else 0.0
    print("%s: worst error / tolerance %.3f" % (what, worst), flush=True)
    assert worst <= 1.0, (what, worst)


def dev(t):
    return None if t is None else t.to(DEV)


def cu_of(lens):
    if lens is None:
        return None, None
    host = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return host.to(DEV), host


# ---- convolution --------------------------------------------------------------------------

CONV = [
    # B, T, D, W, lens, state, bias, silu
    (1, 1, 64, 4, None, False, False, True),
    (2, 3, 64, 4, None, True, True, True),
    (1, 130, 72, 3, None, True, False, True),
    (3, 65, 67, 2, None, False, True, True),          # odd width: one channel a thread
    (1, 200, 520, 4, (0, 1, 2, 64, 0, 3, 130), True, True, True),
    (1, 37, 1000, 4, (37,), True, True, False),
    (1, 66, 5, 3, (1, 1, 64, 0), True, True, True),
    (2, 0, 64, 4, None, True, True, True),            # no tokens at all
]


@pytest.mark.parametrize("pdt", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("c", CONV)
def test_conv(c, dt, pdt):
    B, T, D, W, lens, state, bias, silu = c
    r = gen(hash(c[:4]) % 1000)
    x, w = r(B, T, D).to(dt), (r(D, W) * 0.5).to(pdt)
    b = (r(D) * 0.1).to(pdt) if bias else None
    N = B if lens is None else len(lens)
    init = r(N, W - 1, D).to(dt) if state else None
    dy, dfin = r(B, T, D).to(dt), r(N, W - 1, D).to(dt) if state else None
    cu, host = cu_of(lens)
    xr, wr, br, ir = (None if t is None else R.wide(t).requires_grad_() for t in (x, w, b, init))
    yr, fr = R.conv(xr, wr, br, ir, lens, silu)
    a = (dev(x), dev(w), dev(b))
    y, fin = mixer.conv_fwd(*a, initial_state=dev(init), cu_seqlens=cu, cu_seqlens_host=host, silu=silu)
    # W + 1 terms; silu and its slope are at most 1.1 in size and off by a few ulps
    za = R.conv(xr.detach().abs(), wr.detach().abs(), None if br is None else br.detach().abs(),
                None if ir is None else ir.detach().abs(), lens, False)[0]
    close(y, yr.detach(), za, 16 * 2.0 ** -24, "y")
    assert torch.equal(fin.cpu().double(), fr.detach())
    loss = (yr * R.wide(dy)).sum() + (0 if dfin is None else (fr * R.wide(dfin)).sum())
    leaves = [t for t in (xr, wr, br, ir) if t is not None]
    gr = dict(zip([id(t) for t in leaves], torch.autograd.grad(loss, leaves, allow_unused=True)))
    dx, dw, db, di = mixer.conv_bwd(*a, dev(dy), initial_state=dev(init), d_final_state=dev(dfin), cu_seqlens=cu,
                                    cu_seqlens_host=host, silu=silu, want_d_initial_state=state)
    # sizes: dz <= (1.1 + |z|/4 ...) |dy| <= 2 |dy|; z's own rounding moves silu' by less than its slope, 0.5
    dya = 2 * R.wide(dy).abs() * (1 + za)
    z0 = torch.zeros_like
    xa, wa = xr.detach().abs().requires_grad_(), wr.detach().abs().requires_grad_()
    ba = None if br is None else br.detach().abs().requires_grad_()
    ia = None if ir is None else ir.detach().abs().requires_grad_()
    sa = (R.conv(xa, wa, ba, ia, lens, False)[0] * dya).sum()
    la = [t for t in (xa, wa, ba, ia) if t is not None]
    sl = dict(zip([id(t) for t in la], torch.autograd.grad(sa, la, allow_unused=True)))
    u = 24 * 2.0 ** -24
    for got, t, ta, what in ((dx, xr, xa, "dx"), (dw, wr, wa, "dweight"), (db, br, ba, "dbias"), (di, ir, ia, "dinit")):
        if t is None:
            assert got is None
            continue
        g, s = gr[id(t)], sl[id(ta)]
        m = max(1, B * T) if what in ("dweight", "dbias") else 1
        close(got, z0(t) if g is None else g, z0(t) if s is None else s, u + m * 2.0 ** -24, what)


def test_conv_many_short_sequences_and_many_tokens():
    """200000 sequences of 0 to 2 tokens with a state each, and 5 million tokens: the same, bit for
    bit, as the two halves of them (no sums of the weights' gradients compared there), and a sum
    that is exact in any order."""
    r = gen(31)
    N, D, W = 200000, 64, 4
    lens = torch.randint(0, 3, (N,), generator=torch.Generator().manual_seed(5))
    w, b = dev((r(D, W) * 0.5).to(BF)), dev((r(D) * 0.1).to(BF))

    def go(lens, x, init, dy, dfin):
        host = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)
        k = dict(cu_seqlens=host.to(DEV), cu_seqlens_host=host)
        y, fin = mixer.conv_fwd(x, w, b, initial_state=init, **k)
        dx, dw, db, di = mixer.conv_bwd(x, w, b, dy, initial_state=init, d_final_state=dfin, **k)
        return (y, dx), (fin, di)

    T, h = int(lens.sum()), int(lens[:N // 2].sum())
    x, dy = dev(r(1, T, D).to(BF)), dev(r(1, T, D).to(BF))
    init, dfin = dev(r(N, W - 1, D).to(BF)), dev(r(N, W - 1, D).to(BF))
    whole = go(lens, x, init, dy, dfin)
    halves = (go(lens[:N // 2], x[:, :h].contiguous(), init[:N // 2], dy[:, :h].contiguous(), dfin[:N // 2]),
              go(lens[N // 2:], x[:, h:].contiguous(), init[N // 2:], dy[:, h:].contiguous(), dfin[N // 2:]))
    for i in (0, 1):
        assert torch.equal(whole[0][i], torch.cat([v[0][i] for v in halves], 1))
        assert torch.equal(whole[1][i], torch.cat([v[1][i] for v in halves], 0))

    # no SiLU, x and dy of ones: dweight counts tokens, below 2^24
    T = 5000000
    x = torch.ones(1, T, 2, dtype=BF, device=DEV)
    w2 = torch.ones(2, 2, dtype=F32, device=DEV)
    dx, dw, db, _ = mixer.conv_bwd(x, w2, torch.zeros(2, dtype=F32, device=DEV), x, silu=False)
    assert dw.tolist() == [[T - 1.0, T], [T - 1.0, T]] and db.tolist() == [T, T]
    assert bool((dx[0, :-1] == 2).all()) and bool((dx[0, -1] == 1).all())


def test_conv_slice_of_a_wider_tensor():
    r = gen(5)
    whole = r(2, 50, 96).to(BF).to(DEV)
    w = r(64, 4).to(BF).to(DEV)
    part = whole[:, :, 16:80]
    y, fin = mixer.conv_fwd(part, w)
    y2, fin2 = mixer.conv_fwd(part.contiguous(), w)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    dy = r(2, 50, 64).to(BF).to(DEV)
    for p, q in zip(mixer.conv_bwd(part, w, None, dy), mixer.conv_bwd(part.contiguous(), w, None, dy)):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R_,S,D,W", [(1, 1, 64, 4), (5, 9, 67, 3), (7, 7, 520, 2), (300, 310, 33, 4)])
def test_conv_step(R_, S, D, W, dt):
    r = gen(R_ + D)
    x, state, w, b = r(R_, D).to(dt), r(S, W - 1, D).to(dt), (r(D, W) * 0.5).to(dt), r(D).to(dt)
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(3))[:R_].to(torch.int32)
    if R_ > 4:
        slots[3] = -1                                  # padding
        slots[4] = slots[0]                            # a sequence's next token
    order = state.clone()
    ref, slack = torch.zeros(R_, D, dtype=torch.float64), torch.zeros(R_, D, dtype=torch.float64)
    for i in range(R_):
        s = int(slots[i])
        if s < 0:
            continue
        one = (x[i][None, None], w, b, order[s][None])
        ref[i] = R.conv(*(R.wide(t) for t in one), None)[0][0, 0]
        slack[i] = R.conv(*(R.wide(t).abs() for t in one), None, False)[0][0, 0]
        order[s] = torch.cat([order[s][1:], x[i][None]])
    ds, out = dev(state), torch.full((S, W - 1, D), 7.0, dtype=dt, device=DEV)
    y = mixer.conv_step(dev(x), ds, dev(w), dev(b), slots=dev(slots), state_out=out)
    close(y, ref, slack, 16 * 2.0 ** -24, "y")
    used = sorted({int(s) for s in slots if s >= 0})
    rest = [s for s in range(S) if s not in used]
    assert torch.equal(out.cpu()[used], order[used]) and bool((out.cpu()[rest] == 7.0).all())
    assert torch.equal(ds.cpu(), state)
    y2 = mixer.conv_step(dev(x), ds, dev(w), dev(b), slots=dev(slots))         # in place
    assert torch.equal(y, y2) and torch.equal(ds.cpu(), order)


# ---- selective scan -----------------------------------------------------------------------

def ssm_inputs(seed, B, T, H, G, n, p, dt, pdt, lens, state, ddt=None):
    r = gen(seed)
    N = B if lens is None else len(lens)
    act = torch.nn.functional.silu
    d = dict(x=act(r(B, T, H, p)).to(dt), dt=(r(B, T, H) * 0.5).to(ddt or dt), B=act(r(B, T, G, n)).to(dt),
             C=act(r(B, T, G, n)).to(dt), A=(-(1 + 15 * torch.rand(H, generator=torch.Generator().manual_seed(seed)))).to(pdt),
             D=(1 + 0.1 * r(H)).to(pdt), bias=(r(H) - 2.5).to(pdt), h0=r(N, H, n, p) * 0.3 if state else None,
             dy=r(B, T, H, p).to(dt), dhT=r(N, H, n, p) * 0.3 if state else None)
    return d


def ssm_ref(d, lens, G, softplus=True):
    """Outputs, gradients and the sizes of what they are sums of."""
    H = d["x"].shape[2]
    def go(absolute):
        w = {k: R.wide(t) for k, t in d.items()}
        if absolute:
            w = {k: None if t is None else t.abs() if k not in ("A", "dt", "bias") else t for k, t in w.items()}
        w["B"], w["C"] = (w[k].repeat_interleave(H // G, 2) for k in "BC")
        names = [k for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0") if w[k] is not None]
        for k in names:
            w[k].requires_grad_()
        y, hT = R.ssm(w["x"], w["dt"], w["A"], w["B"], w["C"], w["D"], w["bias"], w["h0"], lens, softplus)
        loss = (y * w["dy"]).sum() + (0 if w["dhT"] is None else (hT * w["dhT"]).sum())
        grads = torch.autograd.grad(loss, [w[k] for k in names], allow_unused=True)
        g = {k: torch.zeros_like(w[k]) if v is None else v for k, v in zip(names, grads)}
        flow = (w["C"] * g["C"]).sum(-1).abs() + (w["B"] * g["B"]).sum(-1).abs()      # [B, T, H], per head
        xdu = (w["x"] * g["x"]).sum(-1).abs()
        for k in "BC":
            g[k] = g[k].unflatten(2, (G, H // G)).sum(3)
        return y.detach(), hT.detach(), g, flow.detach(), xdu.detach()
    return go(False), go(True)


SSM = [
    # B, T, H, G, n, p, lens, state, segment_chunks
    (1, 1, 1, 1, 64, 64, None, False, 0),
    (2, 63, 2, 1, 64, 64, None, True, 0),
    (1, 64, 2, 2, 128, 64, None, True, 0),
    (1, 65, 2, 1, 64, 128, None, True, 0),
    (2, 200, 4, 2, 128, 128, None, True, 1),
    (1, 333, 3, 1, 128, 64, None, False, 2),
    (1, 300, 2, 1, 128, 128, (0, 1, 63, 0, 130, 64, 42, 0), True, 1),
    (1, 300, 4, 4, 64, 64, (100, 200), True, 0),
    (1, 5, 2, 1, 64, 64, (0, 0, 5), True, 0),
    (2, 0, 2, 1, 64, 64, None, True, 0),
]


@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, F32), (F32, F32, F32)])
@pytest.mark.parametrize("c", SSM)
def test_ssm(c, types):
    B, T, H, G, n, p, lens, state, seg = c
    dt, ddt, pdt = types
    d = ssm_inputs(T + H, B, T, H, G, n, p, dt, pdt, lens, state, ddt)
    (y, hT, g, flow, xdu), (ya, hTa, ga, flowa, xdua) = ssm_ref(d, lens, G)
    cu, host = cu_of(lens)
    a = tuple(dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias"))
    gy, gh = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]), cu_seqlens=cu, cu_seqlens_host=host, segment_chunks=seg)
    # one product: bf16 pairs 2^-16, fp32 2^-24; sums of n + 64 products, the decays' exponents
    # (|U| <= a few tens where they matter) and delta, a few ulps each
    prod = (2.0 ** -16 if dt == BF else 0.0) + 64 * 2.0 ** -24
    close(gy, y, ya, prod + (2.0 ** -8 if dt == BF else 0.0), "y")
    close(gh, hT, hTa, 64 * 2.0 ** -24, "final_state")
    dx, dd, dA, dB, dC, dD, db, dh = mixer.ssm_bwd(*a, dev(d["dy"]), initial_state=dev(d["h0"]), d_final_state=dev(d["dhT"]),
                                                   cu_seqlens=cu, cu_seqlens_host=host, segment_chunks=seg,
                                                   want_d_initial_state=state)
    close(dx, g["x"], ga["x"], 2 * prod, "dx")
    close(dB, g["B"], ga["B"], 2 * prod, "dB")
    close(dC, g["C"], ga["C"], 2 * prod, "dC")
    if state:
        close(dh, g["h0"], ga["h0"], 64 * 2.0 ** -24, "d_initial_state")
    # dD: a plain fp32 sum per token and head, fp64 over tokens
    close(dD, g["D"], (d["dy"].double() * d["x"].double()).abs().sum((0, 1, 3)), 64 * 2.0 ** -24, "dD")
    # the gates: sums of flows over a sequence, each flow off by prod of its size
    A = R.wide(d["A"]).abs()
    raw = R.wide(d["dt"]) + R.wide(d["bias"])
    delta, slope = torch.nn.functional.softplus(raw), torch.sigmoid(raw)
    size_da = torch.zeros_like(flowa)
    for i, (r, t0, t1) in enumerate(R.pieces(B, T, lens)):
        extra = 0 if d["dhT"] is None else (hTa[i] * R.wide(d["dhT"][i]).abs()).sum((-1, -2))
        size_da[r, t0:t1] = flowa[r, t0:t1].sum(0) + extra
    size_dt = (xdua / delta + A * size_da) * slope
    close(dd, g["dt"], size_dt, 4 * prod, "ddt")
    close(db, g["bias"], size_dt.sum((0, 1)), 4 * prod, "ddt_bias")
    close(dA, g["A"], (delta * size_da).sum((0, 1)), 4 * prod, "dA")
    if dt == F32:
        # fp32 tensors' flows are summed in fp64, so what counts is what crosses each decay (the
        # absolute run's own gradient), not all that flows: the states, fp32 sums, and the gates
        close(dA, g["A"], ga["A"], 64 * 2.0 ** -24, "dA, of the flows across")


@pytest.mark.parametrize("dt", [BF, F32])
def test_ssm_strong_decay_and_positive_A(dt):
    """A head whose state is gone within a chunk, one that hardly decays, and one that grows
    (A > 0, slightly)."""
    B, T, H, G, n, p = 1, 1300, 3, 1, 64, 64
    d = ssm_inputs(77, B, T, H, G, n, p, dt, F32, None, True, F32)
    d["A"] = torch.tensor([-16.0, -1e-3, 1e-3])
    d["bias"] = torch.tensor([2.0, -3.0, -3.0])
    a = tuple(dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias"))
    w = {k: R.wide(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0")}
    e = lambda t: t.expand(-1, -1, H, -1)  # noqa: E731
    ref, hr = R.ssm(w["x"], w["dt"], w["A"], e(w["B"]), e(w["C"]), w["D"], w["bias"], w["h0"], None)
    ra, ha = R.ssm(w["x"].abs(), w["dt"], w["A"], e(w["B"]).abs(), e(w["C"]).abs(), w["D"], w["bias"], w["h0"].abs(), None)
    prod = (2.0 ** -8 if dt == BF else 0.0) + 128 * 2.0 ** -24
    for seg in (0, 4, 100):
        y, h = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]), segment_chunks=seg)
        close(y, ref, ra, prod, "y, segments of %d" % seg)
        close(h, hr, ha, 128 * 2.0 ** -24, "state, segments of %d" % seg)


@pytest.mark.parametrize("dt", [BF, F32])
def test_ssm_keeps_what_is_small_and_what_is_not_a_number(dt):
    """Inputs at the first tokens only: the state is them, times 2^-60 a segment, and not zero;
    and a NaN among them is in its column of every state and output that follows."""
    B, T, H, G, n, p = 1, 320, 2, 1, 64, 64
    d = ssm_inputs(79, B, T, H, G, n, p, dt, F32, None, False, F32)
    d["x"][:, 4:] = 0
    d["A"], d["dt"] = torch.tensor([-1.0, -1.0]), torch.full((B, T, H), 60 / 256 * 0.6931472)
    w = {k: R.wide(d[k]) for k in ("x", "dt", "A", "B", "C", "D")}
    e = lambda t: t.expand(-1, -1, H, -1)  # noqa: E731
    ref, hr = R.ssm(w["x"], w["dt"], w["A"], e(w["B"]), e(w["C"]), w["D"], None, None, None, False)
    ra, ha = R.ssm(w["x"].abs(), w["dt"], w["A"], e(w["B"]).abs(), e(w["C"]).abs(), w["D"], None, None, None, False)
    assert 2.0 ** -80 < float(hr.abs().max()) < 2.0 ** -70
    a = [dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D")]
    for seg in (0, 1, 4, 100):
        y, h = mixer.ssm_fwd(*a, dt_softplus=False, segment_chunks=seg)
        close(y, ref, ra, (2.0 ** -8 if dt == BF else 0.0) + 128 * 2.0 ** -24, "y, segments of %d" % seg)
        close(h, hr, ha, 128 * 2.0 ** -24, "state, segments of %d" % seg)
    a[0][0, 0, 0, 5] = float("nan")
    for seg in (0, 1, 4, 100):
        y, h = mixer.ssm_fwd(*a, dt_softplus=False, segment_chunks=seg)
        assert torch.isnan(y[0, :, 0, 5]).all() and torch.isnan(h[0, 0, :, 5]).all()
        y[0, :, 0, 5], h[0, 0, :, 5] = 0, 0
        assert torch.isfinite(y).all() and torch.isfinite(h).all()


def test_ssm_options_without_params_and_slices():
    """No D, no dt_bias, no softplus (dt >= 0), x, B and C slices of one tensor."""
    r = gen(11)
    B, T, H, G, n, p = 1, 150, 2, 1, 64, 64
    whole = torch.nn.functional.silu(r(B, T, H * p + 2 * G * n)).to(BF).to(DEV)
    x = whole[..., :H * p].unflatten(-1, (H, p))
    Bm = whole[..., H * p:H * p + G * n].unflatten(-1, (G, n))
    C = whole[..., H * p + G * n:].unflatten(-1, (G, n))
    dt, A = torch.rand(B, T, H).to(DEV) * 0.1, torch.tensor([-1.0, -4.0], device=DEV)
    y, h = mixer.ssm_fwd(x, dt, A, Bm, C, dt_softplus=False)
    y2, h2 = mixer.ssm_fwd(x.contiguous(), dt, A, Bm.contiguous(), C.contiguous(), dt_softplus=False)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    w = [R.wide(t) for t in (x, dt, A, Bm, C)]
    ref, hr = R.ssm(w[0], w[1], w[2], w[3].expand(-1, -1, H, -1), w[4].expand(-1, -1, H, -1), None, None, None, None, False)
    refa = R.ssm(w[0].abs(), w[1], w[2], w[3].abs().expand(-1, -1, H, -1), w[4].abs().expand(-1, -1, H, -1), None, None, None,
                 None, False)
    close(y, ref, refa[0], 2.0 ** -8 + 2.0 ** -16 + 64 * 2.0 ** -24, "y")
    close(h, hr, refa[1], 64 * 2.0 ** -24, "state")
    dy = r(B, T, H, p).to(BF).to(DEV)
    g1 = mixer.ssm_bwd(x, dt, A, Bm, C, None, None, dy, dt_softplus=False)
    g2 = mixer.ssm_bwd(x.contiguous(), dt, A, Bm.contiguous(), C.contiguous(), None, None, dy, dt_softplus=False)
    assert g1[5] is None and g1[6] is None
    for a, b in zip(g1, g2):
        assert (a is None and b is None) or torch.equal(a, b)


def test_ssm_state_carries_over():
    """A prompt in two calls, the second from the first one's state, and then token by token,
    is the prompt in one call."""
    d = ssm_inputs(21, 1, 200, 4, 2, 128, 64, F32, F32, None, True)
    a = [dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias")]
    cut = lambda t0, t1: [a[0][:, t0:t1].contiguous(), a[1][:, t0:t1].contiguous(), a[2], a[3][:, t0:t1].contiguous(),  # noqa: E731
                          a[4][:, t0:t1].contiguous(), a[5], a[6]]
    y, h = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]))
    y1, h1 = mixer.ssm_fwd(*cut(0, 100), initial_state=dev(d["h0"]))
    y2, h2 = mixer.ssm_fwd(*cut(100, 190), initial_state=h1)
    got, state = [y1, y2], h2.clone()
    for t in range(190, 200):
        x, dt, A, B, C, D, bias = cut(t, t + 1)
        got.append(mixer.ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], state, D, bias)[:, None])
    # each part is off by at most the fp32 tolerance of test_ssm
    far = (torch.cat(got, 1) - y).abs().max() / y.abs().max()
    assert float(far) < 2 * 64 * 2.0 ** -24 * 8
    assert float((state - h).abs().max() / h.abs().max()) < 2 * 64 * 2.0 ** -24


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R_,S,H,G,n,p", [(1, 1, 1, 1, 64, 64), (5, 8, 4, 2, 128, 64), (6, 6, 3, 1, 64, 128), (270, 280, 2, 2, 128, 128)])
def test_recurrent_steps(R_, S, H, G, n, p, dt, delta):
    r = gen(R_ + H)
    state = r(S, H, n, p) * 0.3
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(4))[:R_].to(torch.int32)
    if R_ > 4:
        slots[1] = S + 5                               # padding
        slots[4] = slots[0]
    if delta:
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
        q, k, v = unit(r(R_, H, n)).to(dt), unit(r(R_, H, n)).to(dt), r(R_, H, p).to(dt)
        g, beta = torch.nn.functional.logsigmoid(r(R_, H) + 3), torch.sigmoid(r(R_, H)).to(dt)
    else:
        d = ssm_inputs(R_, 1, R_, H, G, n, p, dt, F32, None, False)
    order = R.wide(state).clone()
    ref = torch.zeros(R_, H, p, dtype=torch.float64)
    for i in range(R_):
        s = int(slots[i])
        if not 0 <= s < S:
            continue
        if delta:
            ref[i], order[s] = R.delta_rule(R.wide(q[i]), R.wide(k[i]), R.wide(v[i]), R.wide(g[i]), R.wide(beta[i]), order[s], 0.25)
        else:
            w = {k_: R.wide(d[k_]) for k_ in ("x", "dt", "A", "B", "C", "D", "bias")}
            yy, hh = R.ssm(w["x"][:, i:i + 1], w["dt"][:, i:i + 1], w["A"], w["B"][:, i:i + 1].repeat_interleave(H // G, 2),
                           w["C"][:, i:i + 1].repeat_interleave(H // G, 2), w["D"], w["bias"], order[s][None], None)
            ref[i], order[s] = yy[0, 0], hh[0]
    ds, out = dev(state), torch.full((S, H, n, p), 7.0, device=DEV)
    def call(st, so):
        if delta:
            return mixer.delta_step(*(dev(t) for t in (q, k, v, g, beta)), st, scale=0.25, slots=dev(slots), state_out=so)
        a = [dev(d[k_][0] if k_ in ("x", "dt", "B", "C") else d[k_]) for k_ in ("x", "dt", "A", "B", "C", "D", "bias")]
        return mixer.ssm_step(*a[:5], st, a[5], a[6], slots=dev(slots), state_out=so)
    y = call(ds, out)
    # sums of n products of size |q| |h|: bounded by |q|_1 max |h| <= n * 4 * 2
    close(y, ref, torch.full_like(ref, float(n)), 16 * 2.0 ** -24, "y")
    used = sorted({int(s) for s in slots if 0 <= s < S})
    rest = [s for s in range(S) if s not in used]
    close(out.cpu()[used], order[used], torch.full_like(order[used], 16.0), 16 * 2.0 ** -24, "state")
    assert bool((out.cpu()[rest] == 7.0).all()) and torch.equal(ds.cpu(), state)
    y2 = call(ds, None)
    assert torch.equal(y, y2) and torch.equal(ds.cpu()[used], out.cpu()[used]) and torch.equal(ds.cpu()[rest], state[rest])


def test_delta_step_continues_chunk_fwd():
    """A prompt's final state from chunk_fwd, continued by single tokens, is the longer prompt."""
    r = gen(31)
    B, T, H, D = 2, 140, 3, 128
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = (t.to(DEV) for t in (unit(r(B, T, H, D)), unit(r(B, T, H, D)), r(B, T, H, D)))
    g, beta = torch.nn.functional.logsigmoid(r(B, T, H) + 3).to(DEV), torch.sigmoid(r(B, T, H)).to(DEV)
    o, h = binding.chunk_fwd(q, k, v, g, beta)
    c = lambda t: t[:, :130].contiguous()  # noqa: E731
    _, state = binding.chunk_fwd(c(q), c(k), c(v), c(g), c(beta))
    for t in range(130, T):
        ot = mixer.delta_step(*(u[:, t].contiguous() for u in (q, k, v, g, beta)), state)
        # chunk_fwd's own fp32 bar against the 64-bit oracle is 1e-5
        assert float((ot - o[:, t]).norm() / o[:, t].norm()) < 2e-5
    assert float((state - h).norm() / h.norm()) < 2e-5


# ---- norm ---------------------------------------------------------------------------------

NORM = [
    # rows, H, D, affine, gate
    (1, 1, 1, True, False),
    (3, 1, 64, True, True),
    (50, 4, 128, True, True),
    (33, 5, 96, True, False),
    (20, 3, 67, True, True),
    (70, 1, 2048, True, False),
    (40, 1, 3001, True, True),
    (9, 1, 8192, False, False),
    (5, 1, 8191, True, True),
    (200, 2, 256, False, True),
    (17, 1, 512, True, True),
    (0, 2, 64, True, True),
]


@pytest.mark.parametrize("pdt", [BF, F32])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("c", NORM)
def test_norm(c, dt, pdt):
    rows, H, D, affine, gate = c
    r = gen(rows + D)
    shape = (rows, H, D) if H > 1 else (rows, D)
    par = (H, D) if H > 1 else (D,)
    x = (r(*shape) * 1.5 + 3).to(dt)
    w, b = ((1 + 0.1 * r(*par)).to(pdt), (0.1 * r(*par)).to(pdt)) if affine else (None, None)
    z = r(*shape).to(dt) if gate else None
    dy = r(*shape).to(dt)
    eps = 1e-5
    xr, wr, br, zr = (None if t is None else R.wide(t).requires_grad_() for t in (x, w, b, z))
    yr, mr, rr = R.norm(xr, wr, br, zr, eps)
    y, mean, rstd = mixer.norm_fwd(dev(x), dev(w), dev(b), gate=dev(z), eps=eps)
    u = 2.0 ** -24
    # mean and variance: sums in a tree of depth <= 6 + 8 over at most 32 terms a lane
    xm = xr.detach().abs().mean(-1)
    close(mean, mr.detach(), xm, 48 * u, "mean")
    # rstd: x - mean is off by (48 + 2) u of |x|'s size, relative to the deviation 1 / rstd
    kappa = 1 + xm * rr.detach()
    close(rstd, rr.detach(), rr.detach() * kappa, 64 * u, "rstd")
    size = (xr.detach().abs() + xm[..., None]) * rr.detach()[..., None]
    ysz = size * kappa[..., None] * (1 if w is None else wr.detach().abs()) + (0 if b is None else br.detach().abs())
    if gate:
        ysz = ysz * (1 + zr.detach().abs())
    close(y, yr.detach(), ysz, 80 * u, "y")
    leaves = [t for t in (xr, wr, br, zr) if t is not None]
    gr = dict(zip([id(t) for t in leaves], torch.autograd.grad((yr * R.wide(dy)).sum(), leaves)))
    dx, dw, db, dz = mixer.norm_bwd(dev(x), mean, rstd, dev(dy), dev(w), dev(b), gate=dev(z))
    # sizes of the summands, everything absolute
    dn = R.wide(dy).abs() * (1 if z is None else 1 + zr.detach().abs())
    g = dn * (1 if w is None else wr.detach().abs())
    big = kappa[..., None] * size                                   # |xh| and what its rounding scales with
    if rows:
        xsz = rr.detach()[..., None] * kappa[..., None] * (g + g.mean(-1, keepdim=True) + big * (g * big).mean(-1, keepdim=True))
    else:
        xsz = torch.zeros(shape, dtype=torch.float64)
    close(dx, gr[id(xr)], xsz, 200 * u, "dx")
    m = max(1, rows)
    if affine:
        close(dw, gr[id(wr)], (dn * big).sum(0), (100 + m) * u, "dweight")
        close(db, gr[id(br)], dn.sum(0), (16 + m) * u, "dbias")
    else:
        assert dw is None and db is None
    if gate:
        close(dz, gr[id(zr)], R.wide(dy).abs() * ysz * 2, 100 * u, "dgate")


# ---- together, as a layer runs them -------------------------------------------------------

def mixer_layer(h, P, cu, host):
    """conv -> (x, B, C) -> scan -> gated norm of the heads."""
    T = h.shape[1]
    u, _ = mixer.conv_fwd(h, P["cw"], P["cb"], cu_seqlens=cu, cu_seqlens_host=host)
    H, p, n = P["H"], P["p"], P["n"]
    x = u[..., :H * p].unflatten(-1, (H, p))
    B, C = (u[..., H * p + i * n:H * p + (i + 1) * n].unflatten(-1, (1, n)) for i in (0, 1))
    y, _ = mixer.ssm_fwd(x, P["dt"], P["A"], B, C, P["D"], P["bias"], cu_seqlens=cu, cu_seqlens_host=host)
    o, mean, rstd = mixer.norm_fwd(y.reshape(1, T, H, p), P["nw"], P["nb"], gate=P["z"])
    return u, x, B, C, y, o, mean, rstd


def test_layer_forward_and_backward():
    """Convolution, scan and norm in a run, forward and back, on packed sequences, in fp32,
    against the same layer in 64 bits differentiated by autograd."""
    r = gen(41)
    H, p, n, T, lens = 2, 64, 64, 150, (70, 0, 3, 77)
    D = H * p + 2 * n
    P = dict(H=H, p=p, n=n, cw=r(D, 4) * 0.5, cb=r(D) * 0.1, dt=r(1, T, H) * 0.5, A=-torch.tensor([1.0, 5.0]), D=torch.ones(H),
             bias=r(H) - 2.5, nw=1 + 0.1 * r(H, p), nb=0.1 * r(H, p), z=r(1, T, H, p))
    h, do = r(1, T, D), r(1, T, H, p)
    cu, host = cu_of(lens)
    Q = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in P.items()}
    u, x, B, C, y, o, mean, rstd = mixer_layer(dev(h), Q, cu, host)
    dyn, dnw, dnb, dz = mixer.norm_bwd(y, mean, rstd, dev(do), Q["nw"], Q["nb"], gate=Q["z"])
    dx, ddt, dA, dB, dC, dD, dbias, _ = mixer.ssm_bwd(x, Q["dt"], Q["A"], B, C, Q["D"], Q["bias"], dyn, cu_seqlens=cu,
                                                      cu_seqlens_host=host)
    du = torch.cat([dx.flatten(2), dB.flatten(2), dC.flatten(2)], -1)
    dh, dcw, dcb, _ = mixer.conv_bwd(dev(h), Q["cw"], Q["cb"], du, cu_seqlens=cu, cu_seqlens_host=host)

    w = {k: R.wide(v).requires_grad_() for k, v in P.items() if isinstance(v, torch.Tensor)}
    hr = R.wide(h).requires_grad_()
    ur, _ = R.conv(hr, w["cw"], w["cb"], None, lens)
    xr = ur[..., :H * p].unflatten(-1, (H, p))
    Br, Cr = (ur[..., H * p + i * n:H * p + (i + 1) * n].unflatten(-1, (1, n)).expand(-1, -1, H, -1) for i in (0, 1))
    yr, _ = R.ssm(xr, w["dt"], w["A"], Br, Cr, w["D"], w["bias"], None, lens)
    outr, _, _ = R.norm(yr, w["nw"], w["nb"], w["z"], 1e-5)
    names = ["cw", "cb", "dt", "A", "D", "bias", "nw", "nb", "z"]
    gr = torch.autograd.grad((outr * R.wide(do)).sum(), [hr] + [w[k] for k in names])
    # three operators of fp32 sums of at most a few hundred terms each, relative to the whole
    # tensor (2-norm): 3 * 2^8 * 2^-24
    for what, got, ref in [("out", o, outr.detach()), ("dh", dh, gr[0])] + list(zip(names, (dcw, dcb, ddt, dA, dD, dbias, dnw, dnb, dz), gr[1:])):
        off = float((got.cpu().double() - ref).norm() / ref.norm())
        print("%s: %.2e" % (what, off), flush=True)
        assert off < 3 * 2.0 ** -16, (what, off)


# ---- calls that are not alone on the default stream ---------------------------------------

def everything(seed, n_tokens=200):
    """Every entry point once, on inputs of a seed: a function that makes the calls, and its
    inputs by name (which a test may write over)."""
    r = gen(seed)
    H, G, n, p, T = 4, 2, 64, 128, n_tokens
    lens = (T - 67, 0, 3, 64)
    cu, host = cu_of(lens)
    D = H * p
    d = {k: dev(v) for k, v in ssm_inputs(seed, 1, T, H, G, n, p, BF, F32, lens, True).items()}
    d.update(cw=r(D, 4).to(BF).to(DEV), cx=r(1, T, D).to(BF).to(DEV), cdy=r(1, T, D).to(BF).to(DEV), ci=r(4, 3, D).to(BF).to(DEV),
             nw=r(H, p).to(DEV), nb=r(H, p).to(DEV), z=r(1, T, H, p).to(BF).to(DEV), slots=torch.tensor([3, 0, 3, -1], dtype=torch.int32).to(DEV),
             cs=r(5, 3, D).to(BF).to(DEV), hs=r(5, H, n, p).to(DEV), q=r(4, H, n).to(BF).to(DEV), g=-r(4, H).abs().to(DEV),
             be=torch.sigmoid(r(4, H)).to(BF).to(DEV), cso=torch.zeros(5, 3, D, dtype=BF, device=DEV), hso=torch.zeros(5, H, n, p, device=DEV))

    def run():
        k = dict(cu_seqlens=cu, cu_seqlens_host=host)
        out = list(mixer.conv_fwd(d["cx"], d["cw"], None, initial_state=d["ci"], **k))
        out += mixer.conv_bwd(d["cx"], d["cw"], None, d["cdy"], initial_state=d["ci"], **k)
        a = [d[x] for x in ("x", "dt", "A", "B", "C", "D", "bias")]
        out += mixer.ssm_fwd(*a, initial_state=d["h0"], segment_chunks=1, **k)
        out += mixer.ssm_bwd(*a, d["dy"], initial_state=d["h0"], d_final_state=d["dhT"], segment_chunks=1, **k)
        y, mean, rstd = mixer.norm_fwd(d["x"], d["nw"], d["nb"], gate=d["z"])
        out += [y, mean, rstd, *mixer.norm_bwd(d["x"], mean, rstd, d["dy"], d["nw"], d["nb"], gate=d["z"])]
        one = lambda t: t[0, :4].contiguous()  # noqa: E731
        out.append(mixer.conv_step(one(d["cx"]), d["cs"], d["cw"], slots=d["slots"], state_out=d["cso"]))
        out.append(mixer.ssm_step(one(d["x"]), one(d["dt"]), d["A"], one(d["B"]), one(d["C"]), d["hs"], slots=d["slots"], state_out=d["hso"]))
        out.append(d["hso"].clone())
        out.append(mixer.delta_step(d["q"], d["q"], one(d["x"]), d["g"], d["be"], d["hs"], slots=d["slots"], state_out=d["hso"]))
        return [t for t in out if t is not None] + [d["cso"].clone(), d["hso"].clone()]
    return run, d


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_repeat_bit_for_bit():
    run, _ = everything(51)
    first = run()
    for _ in range(3):
        assert same(first, run())


def test_two_streams_at_once():
    (run1, _), (run2, _) = everything(52), everything(53, 330)
    want1, want2 = run1(), run2()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(s1):
            got1 = run1()
        with torch.cuda.stream(s2):
            got2 = run2()
        torch.cuda.synchronize()
        assert same(want1, got1) and same(want2, got2)


def test_graph_replays_with_new_inputs():
    """A captured run of every entry point, replayed between eager runs and with its inputs
    written over, gives what an eager run on those inputs gives."""
    run, d = everything(54)
    others = [everything(s)[1] for s in (55, 56, 54)]
    run()                                                  # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for new in others:
        for k, t in d.items():
            if t is not None:
                t.copy_(new[k])
        torch.cuda.synchronize()
        want = [t.clone() for t in run()]
        d["cso"].zero_(), d["hso"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, captured)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, captured)


def test_other_sequences_do_not_leak():
    """NaN in one packed sequence stays in it: forward, gradients and final states."""
    lens = (70, 5, 0, 60)
    cu, host = cu_of(lens)
    d = ssm_inputs(61, 1, 135, 2, 1, 64, 64, BF, F32, lens, True)
    r = gen(62)
    cx, cw, cdy = r(1, 135, 24).to(BF), r(24, 4).to(BF), r(1, 135, 24).to(BF)
    bad = slice(70, 75)
    d["x"][:, bad], d["dy"][:, bad], d["B"][:, bad], d["C"][:, bad] = (float("nan"),) * 4
    cx[:, bad], cdy[:, bad] = float("nan"), float("inf")
    k = dict(cu_seqlens=cu, cu_seqlens_host=host)
    a = [dev(d[x]) for x in ("x", "dt", "A", "B", "C", "D", "bias")]
    y, h = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]), **k)
    g = mixer.ssm_bwd(*a, dev(d["dy"]), initial_state=dev(d["h0"]), d_final_state=dev(d["dhT"]), **k)
    cy, cf = mixer.conv_fwd(dev(cx), dev(cw), **k)
    cg = mixer.conv_bwd(dev(cx), dev(cw), None, dev(cdy), **k)
    for t in (y, g[0], g[1], g[3], g[4], cy, cg[0]):
        fine = torch.isfinite(t[0].flatten(1)).all(1).cpu()
        assert bool(fine[:70].all()) and bool(fine[75:].all())
    for t in (h, g[7], cf, cg[3]):
        fine = torch.isfinite(t.flatten(1)).all(1).cpu().tolist()
        assert fine[0] and fine[2] and fine[3]


def test_all_sequences_empty():
    cu, host = cu_of((0, 0, 0))
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    init = torch.randn(3, 3, 16).to(BF).to(DEV)
    y, fin = mixer.conv_fwd(z(1, 0, 16), z(16, 4), initial_state=init, cu_seqlens=cu, cu_seqlens_host=host)
    assert y.shape == (1, 0, 16) and torch.equal(fin, init)
    dx, dw, _, di = mixer.conv_bwd(z(1, 0, 16), z(16, 4), None, z(1, 0, 16), initial_state=init, d_final_state=init, cu_seqlens=cu,
                                   cu_seqlens_host=host)
    assert torch.equal(di, init) and not bool(dw.any())
    h0 = torch.randn(3, 2, 64, 64).to(DEV)
    a = (z(1, 0, 2, 64), z(1, 0, 2), -torch.ones(2, device=DEV), z(1, 0, 1, 64), z(1, 0, 1, 64), None, None)
    y, h = mixer.ssm_fwd(*a, initial_state=h0, cu_seqlens=cu, cu_seqlens_host=host)
    assert y.shape == (1, 0, 2, 64) and torch.equal(h, h0)
    g = mixer.ssm_bwd(*a, z(1, 0, 2, 64), initial_state=h0, d_final_state=2 * h0, cu_seqlens=cu, cu_seqlens_host=host)
    assert torch.equal(g[7], 2 * h0) and not bool(g[2].any())


def test_nothing_crosses_the_first_decay():
    """Single tokens from a zero state: the gradient of A is zero, and ddt only x . du."""
    d = ssm_inputs(71, 3, 1, 2, 1, 64, 64, BF, F32, None, False)
    a = [dev(d[x]) for x in ("x", "dt", "A", "B", "C", "D", "bias")]
    g = mixer.ssm_bwd(*a, dev(d["dy"]))
    assert not bool(g[2].any()) and bool(g[1].abs().sum() > 0)


@pytest.mark.parametrize("op", ["conv", "ssm", "norm"])
def test_gradients_are_the_differences(op):
    """Directional derivatives of the fp32 kernels by central differences of their own outputs.
    An output's fp32 rounding (2^-24 of |y|, some tens of them in a sum) over a step of 2^-6
    bounds the noise; the third derivative's term is 2^-12 / 6 of a size near the loss's."""
    r = gen(81)
    cu, host = cu_of((50, 3, 20))
    if op == "conv":
        leaves = [r(1, 73, 32), r(32, 4) * 0.5, r(32) * 0.1]
        do = [r(1, 73, 32)]
        f = lambda x, w, b: mixer.conv_fwd(x, w, b, cu_seqlens=cu, cu_seqlens_host=host)[:1]  # noqa: E731
        back = lambda x, w, b: mixer.conv_bwd(x, w, b, dev(do[0]), cu_seqlens=cu, cu_seqlens_host=host)[:3]  # noqa: E731
    elif op == "ssm":
        d = ssm_inputs(82, 1, 73, 2, 1, 64, 64, F32, F32, (50, 3, 20), True)
        leaves = [d[k] for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0")]
        do = [r(1, 73, 2, 64), r(3, 2, 64, 64) * 0.3]
        f = lambda x, dt, A, B, C, D, b, h: mixer.ssm_fwd(x, dt, A, B, C, D, b, initial_state=h, cu_seqlens=cu, cu_seqlens_host=host)  # noqa: E731
        back = lambda x, dt, A, B, C, D, b, h: mixer.ssm_bwd(x, dt, A, B, C, D, b, dev(do[0]), initial_state=h, d_final_state=dev(do[1]),  # noqa: E731
                                                             cu_seqlens=cu, cu_seqlens_host=host)
    else:
        leaves = [r(40, 3, 48) + 1, r(3, 48), r(3, 48), r(40, 3, 48)]
        do = [r(40, 3, 48)]
        f = lambda x, w, b, z: mixer.norm_fwd(x, w, b, gate=z)[:1]  # noqa: E731
        def back(x, w, b, z):
            _, mean, rstd = mixer.norm_fwd(x, w, b, gate=z)
            return mixer.norm_bwd(x, mean, rstd, dev(do[0]), w, b, gate=z)
    leaves = [dev(t) for t in leaves]
    loss = lambda ts: sum(float((y.double() * dev(w).double()).sum()) for y, w in zip(f(*ts), do))  # noqa: E731
    grads = back(*leaves)
    size = sum(float((y.double().abs() * dev(w).double().abs()).sum()) for y, w in zip(f(*leaves), do))
    step = 2.0 ** -6
    for i, (t, g) in enumerate(zip(leaves, grads)):
        v = dev(gen(90 + i)(*t.shape))
        v = v / v.norm()
        at = lambda e: loss([u + e * v if j == i else u for j, u in enumerate(leaves)])  # noqa: E731
        diff = (at(step) - at(-step)) / (2 * step)
        want = float((g.double() * v.double()).sum())
        print("%s leaf %d: %.6g by differences, %.6g" % (op, i, diff, want), flush=True)
        assert abs(diff - want) < size * (32 * 2.0 ** -24 / step + step * step / 6) + 1e-3 * abs(want), (op, i)
