"""The operators of gated_deltanet_chunked_fwd_amd.mixer on the GPU where their bounds are
tight: results whose sums nearly cancel, sizes that take every branch of the kernels, values
that are not finite.  References and tolerances as in test_gpu_mixer.py."""
import pytest
import torch

from gated_deltanet_chunked_fwd_amd import mixer
from tests import mixer_ref as R
from tests.test_gpu_mixer import BF, F32, close, cu_of, dev, gen, ssm_inputs, ssm_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seg", [0, 2])
@pytest.mark.parametrize("n,p", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_ssm_outputs_of_a_long_memory(n, p, seg):
    """bf16 outputs that are nearly all C h, with products of both signs: the state enters as a
    bf16 pair, which leaves 2^-8 of 2^-8 of each product, as the pair of the q k products
    does; 128 more fp32 roundings for the sums and the decays."""
    B, T, H = 1, 200, 2
    d = ssm_inputs(n + p, B, T, H, 1, n, p, BF, F32, None, True, F32)
    d["C"] = gen(7)(B, T, 1, n).to(BF)
    d["h0"] = d["h0"] * 100
    d["A"] = torch.tensor([-1e-3, -1e-2])
    w = {k: R.wide(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias", "h0")}
    e = lambda t: t.expand(-1, -1, H, -1)  # noqa: E731
    ref, hr = R.ssm(w["x"], w["dt"], w["A"], e(w["B"]), e(w["C"]), w["D"], w["bias"], w["h0"], None)
    ra, ha = R.ssm(w["x"].abs(), w["dt"], w["A"], e(w["B"]).abs(), e(w["C"]).abs(), w["D"], w["bias"], w["h0"].abs(), None)
    a = tuple(dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias"))
    y, h = mixer.ssm_fwd(*a, initial_state=dev(d["h0"]), segment_chunks=seg)
    close(y, ref, ra, 2.0 ** -16 + 128 * 2.0 ** -24, "y")
    close(h, hr, ha, 128 * 2.0 ** -24, "state")


@pytest.mark.parametrize("op", ["conv", "conv_step", "norm"])
def test_silu_of_fp32_tensors(op):
    """SiLU and its slope of fp32 arguments far below zero, where exp(-z) is nearly all of
    them.  Half steps of 2^-24: exp 2 (an ulp), 1 + exp, the division, z times it: 5, and one
    for z.  The slope s (1 + z (1 - s)), |z| >= 10: s 4 half steps, 1 - s and z times it 2,
    one more with |z| / (|z| - 1) <= 1.2 of these, the product and dy times it: 4 + 1.2 * 3
    + 2 < 10."""
    u = 2.0 ** -24
    z = -(10 + 70 * torch.rand(512, 64, generator=torch.Generator().manual_seed(3))).to(F32)
    z64 = z.double()
    s64 = torch.sigmoid(z64)
    silu, slope = z64 * s64, s64 * (1 + z64 * (1 - s64))
    w = torch.tensor([0.0, 1.0]).repeat(64, 1)                # z is the input itself
    if op == "conv":
        y, _ = mixer.conv_fwd(dev(z)[None], dev(w))
        close(y[0], silu, silu.abs(), 5 * u, "y")
        dx, _, _, _ = mixer.conv_bwd(dev(z)[None], dev(w), None, torch.ones(1, 512, 64, device="cuda"))
        close(dx[0], slope, slope.abs(), 9 * u, "dx")
    elif op == "conv_step":
        y = mixer.conv_step(dev(z), torch.zeros(512, 1, 64, device="cuda"), dev(w))
        close(y, silu, silu.abs(), 5 * u, "y")
    else:
        x, dy = gen(4)(512, 64), gen(5)(512, 64)
        plain, mean, rstd = mixer.norm_fwd(dev(x))
        y, _, _ = mixer.norm_fwd(dev(x), gate=dev(z))         # the same values, times the gate's SiLU
        close(y, plain.cpu().double() * silu, (plain.cpu().double() * silu).abs(), 6 * u, "y")
        dz = mixer.norm_bwd(dev(x), mean, rstd, dev(dy), gate=dev(z))[3]
        # (x - mean) rstd is formed again from the same numbers: the bits of `plain`
        ref = plain.cpu().double() * dy.double() * slope
        close(dz, ref, ref.abs(), 11 * u, "dgate")


def check_ssm(B, T, H, G, n, p, lens, seg, types):
    """ssm_fwd and ssm_bwd with start and end states against the 64-bit reference, with
    test_ssm's bounds: one product 2^-16 (bf16 pairs) and 64 fp32 roundings, 128 for
    states carried over this many chunks, flows of the gates by the size of all of them."""
    dt, ddt, pdt = types
    d = ssm_inputs(T + n + seg, B, T, H, G, n, p, dt, pdt, lens, True, ddt)
    (y, hT, g, flow, xdu), (ya, hTa, ga, flowa, xdua) = ssm_ref(d, lens, G)
    cu, host = cu_of(lens)
    a = tuple(dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias"))
    k = dict(initial_state=dev(d["h0"]), cu_seqlens=cu, cu_seqlens_host=host, segment_chunks=seg)
    gy, gh = mixer.ssm_fwd(*a, **k)
    prod = (2.0 ** -16 if dt == BF else 0.0) + 128 * 2.0 ** -24
    close(gy, y, ya, prod, "y")
    close(gh, hT, hTa, 128 * 2.0 ** -24, "final_state")
    dx, dd, dA, dB, dC, dD, db, dh = mixer.ssm_bwd(*a, dev(d["dy"]), d_final_state=dev(d["dhT"]), **k)
    close(dx, g["x"], ga["x"], 2 * prod, "dx")
    close(dB, g["B"], ga["B"], 2 * prod, "dB")
    close(dC, g["C"], ga["C"], 2 * prod, "dC")
    close(dh, g["h0"], ga["h0"], 128 * 2.0 ** -24, "d_initial_state")
    close(dD, g["D"], (d["dy"].double() * d["x"].double()).abs().sum((0, 1, 3)), 64 * 2.0 ** -24, "dD")
    A, raw = R.wide(d["A"]).abs(), R.wide(d["dt"]) + R.wide(d["bias"])
    delta, slope = torch.nn.functional.softplus(raw), torch.sigmoid(raw)
    size_da = torch.zeros_like(flowa)
    for i, (r, t0, t1) in enumerate(R.pieces(B, T, lens)):
        size_da[r, t0:t1] = flowa[r, t0:t1].sum(0) + (hTa[i] * R.wide(d["dhT"][i]).abs()).sum((-1, -2))
    size_dt = (xdua / delta + A * size_da) * slope
    close(dd, g["dt"], size_dt, 4 * prod, "ddt")
    close(db, g["bias"], size_dt.sum((0, 1)), 4 * prod, "ddt_bias")
    close(dA, g["A"], (delta * size_da).sum((0, 1)), 4 * prod, "dA")
    # The bounds above are of all that flows, hundreds of times what is left of it.  Of the result
    # itself, in the 2-norm: ddt takes a sum of the flows behind it in its segment, at most
    # 64 * 16 (the longest segment there is), each some 8 times what crosses one decay and off by a
    # few times 2^-24 of itself: sqrt(1024) * 8 * 4 * 2^-24 = 2^-14 (fp32 tensors are summed in fp64:
    # the states' 2^-24 are left).  ddt_bias and dA add up ddt's errors, which have one sign over a
    # segment, where the values have both: 2^6 times, for 1024 * 2^2 tokens.
    bars = (2.0 ** -14, 2.0 ** -8) if dt == BF else (2.0 ** -20, 2.0 ** -14)
    for got, ref, what, bar in ((dd, g["dt"], "ddt", bars[0]), (db, g["bias"], "ddt_bias", bars[1]), (dA, g["A"], "dA", bars[1])):
        off = float((got.cpu().double() - ref).norm() / ref.norm())
        print("%s: %.2e of the result" % (what, off), flush=True)
        assert off < bar, (what, off)


@pytest.mark.parametrize("types", [(BF, F32, F32), (F32, F32, F32)])
@pytest.mark.parametrize("n,p,seg", [(64, 64, 1), (64, 64, 3), (64, 64, 5), (64, 64, 12), (64, 64, 100), (64, 64, 0),
                                     (128, 64, 5), (64, 128, 12), (128, 128, 100)])
def test_ssm_segments_of_any_length(n, p, seg, types):
    """21 chunks, the last one ragged: more segments than the chain over them reads ahead (1,
    3), and gates' gradients of four waves (3) and of eight in one round (5), in two of
    which the last is partial (12) or whole (100: segments of 16 chunks there, one forward)."""
    check_ssm(1, 1300, 2, 1, n, p, None, seg, types)


@pytest.mark.parametrize("types", [(BF, F32, F32), (F32, F32, F32)])
@pytest.mark.parametrize("seg", [0, 1])
def test_ssm_more_sequences_than_a_wave_has_lanes(seg, types):
    """150 packed sequences, empty, of single tokens and of several segments around the 64th
    and 128th."""
    lens = [(0, 1, 3, 17)[i % 4] for i in range(150)]
    for i, v in ((5, 130), (62, 0), (63, 200), (64, 65), (65, 0), (126, 129), (127, 0), (128, 66), (149, 70)):
        lens[i] = v
    check_ssm(1, sum(lens), 2, 2, 64, 64, tuple(lens), seg, types)


def test_views_that_start_anywhere():
    """slots, gates, cu_seqlens and statistics that start on an element give what aligned copies
    give, and nothing around them is read or written."""
    def shifted(t):
        room = torch.full((t.numel() + 17,), 3, dtype=t.dtype, device="cuda")
        v = room[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16
        return v
    lens = (70, 0, 3, 77)
    d = {k: dev(v) for k, v in ssm_inputs(91, 1, 150, 3, 1, 64, 64, BF, F32, lens, True).items()}
    cu, host = cu_of(lens)
    slots = dev(torch.tensor([3, 0, 3, -1], dtype=torch.int32))
    r = gen(92)
    state, cs = dev(r(5, 3, 64, 64)), dev(r(5, 3, 192).to(BF))
    g, beta = dev(-r(4, 3).abs()), dev(torch.sigmoid(r(4, 3)).to(BF))
    one = lambda t: t[0, :4].contiguous()  # noqa: E731

    def run(f):
        a = [d["x"], f(d["dt"]), f(d["A"]), d["B"], d["C"], f(d["D"]), f(d["bias"])]
        k = dict(initial_state=d["h0"], cu_seqlens=f(cu), cu_seqlens_host=host)
        out = [*mixer.ssm_fwd(*a, **k), *mixer.ssm_bwd(*a, d["dy"], d_final_state=d["dhT"], **k)]
        x = d["x"].flatten(2)
        w = dev(torch.ones(192, 4)).to(BF)
        out += [*mixer.conv_fwd(x, w, cu_seqlens=f(cu), cu_seqlens_host=host)]
        y, mean, rstd = mixer.norm_fwd(d["x"], gate=d["dy"])
        out += [y, *mixer.norm_bwd(d["x"], f(mean), f(rstd), d["dy"], gate=d["dy"])]
        h, c = state.clone(), cs.clone()
        out += [mixer.ssm_step(one(d["x"]), f(one(d["dt"])), f(d["A"]), one(d["B"]), one(d["C"]), h, f(d["D"]), f(d["bias"]), slots=f(slots))]
        out += [mixer.delta_step(one(d["x"]), one(d["x"]), one(d["x"]), f(g), f(beta), h, slots=f(slots))]
        out += [mixer.conv_step(one(x), c, w, slots=f(slots)), h, c]
        return [t for t in out if t is not None]
    for a, b in zip(run(lambda t: t), run(shifted)):
        assert torch.equal(a, b)


def test_norm_of_more_rows_than_a_launch_has_workgroups():
    """2^24 + 3 rows of 8 elements, 32 to a workgroup: each as a call on some of them gives it, and
    the weights' gradients against 64 bits (a sum of m fp32 products: m 2^-24 of their
    sizes, far from reached)."""
    rows, D = (1 << 24) + 3, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x, dy = (torch.randn(rows, D, generator=g, device="cuda").to(BF) for _ in range(2))
    w, b = (torch.randn(D, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = mixer.norm_fwd(x, w, b)
    dx, dw, db, _ = mixer.norm_bwd(x, mean, rstd, dy, w, b)
    for part in (slice(0, 64), slice((1 << 24) - 64, rows)):
        p = x[part].contiguous()
        y1, m1, r1 = mixer.norm_fwd(p, w, b)
        assert torch.equal(y[part], y1) and torch.equal(mean[part], m1) and torch.equal(rstd[part], r1)
        assert torch.equal(dx[part], mixer.norm_bwd(p, m1, r1, dy[part].contiguous(), w, b)[0])
    dwr = torch.zeros(D, dtype=torch.float64, device="cuda")
    dbr, size = dwr.clone(), dwr.clone()
    for at in range(0, rows, 1 << 22):
        k = slice(at, at + (1 << 22))
        xh = (x[k].double() - mean[k, None].double()) * rstd[k, None].double()
        dwr += (dy[k].double() * xh).sum(0)
        dbr += dy[k].double().sum(0)
        size += (dy[k].double() * xh).abs().sum(0)
    # in chains of at most 2^14 of a lane, then a tree: 2^-10 of the sizes is 2^14 roundings
    close(dw, dwr.cpu(), size.cpu(), 2.0 ** -10, "dweight")
    close(db, dbr.cpu(), size.cpu(), 2.0 ** -10, "dbias")


@pytest.mark.parametrize("seg", [0, 1, 100])
@pytest.mark.parametrize("dt,n,p", [(BF, 128, 128), (BF, 64, 64), (BF, 128, 64), (BF, 64, 128), (F32, 64, 64), (F32, 128, 128)])
def test_ssm_fwd_never_looks_ahead(dt, n, p, seg):
    """Values that are not finite leave every output before them, and every other column, as it
    is with zeros in their place, bit for bit; from their token on their column is not
    finite.  In B, C and dt they leave the tokens before them as they are."""
    B, T, H = 2, 200, 2
    d = ssm_inputs(95, B, T, H, 1, n, p, dt, F32, None, True, F32)
    a = [dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias")]
    k = dict(initial_state=dev(d["h0"]), segment_chunks=seg)
    where = [(0, 199, 0, 3, float("nan")), (0, 64, 1, 0, float("inf")), (1, 0, 0, p - 1, float("nan")), (1, 63, 1, 17, -float("inf")),
             (1, 70, 0, 2, float("nan")), (1, 101, 0, 2, float("inf")), (0, 15, 0, 8, float("nan")), (0, 48, 0, 9, float("inf"))]
    for b, t, h, c, v in where:
        a[0][b, t, h, c] = 0
    y0, h0 = mixer.ssm_fwd(*a, **k)
    for b, t, h, c, v in where:
        a[0][b, t, h, c] = v
    y, hT = mixer.ssm_fwd(*a, **k)
    first = torch.full((B, 1, H, p), T, device="cuda")
    for b, t, h, c, v in where:
        first[b, 0, h, c] = min(t, int(first[b, 0, h, c]))
    after = torch.arange(T, device="cuda")[None, :, None, None] >= first
    assert torch.equal(y[~after], y0[~after]) and not bool(torch.isfinite(y[after]).any())
    gone = (first < T)[:, 0, :, None, :].expand_as(hT)
    assert torch.equal(hT[~gone], h0[~gone]) and not bool(torch.isfinite(hT[gone]).any())
    for i in (1, 3, 4):
        clean = mixer.ssm_fwd(*[a[0].nan_to_num(0, 0, 0)] + a[1:], **k)[0]
        bad = [t.clone() for t in a]
        bad[0] = bad[0].nan_to_num(0, 0, 0)
        bad[i][:, 90] = float("nan")
        y = mixer.ssm_fwd(*bad, **k)[0]
        assert torch.equal(y[:, :90], clean[:, :90]) and bool(torch.isnan(y[:, 90]).any())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("seg", [0, 1, 100])
def test_ssm_after_a_decay_to_nothing(dt, seg):
    """A token whose decay is exp(-10^12) forgets all before it and leaves what follows as exact as
    ever (test_ssm's bounds), forward and back; and a head of A = -inf has no memory."""
    B, T, H, n, p = 1, 150, 2, 64, 64
    d = ssm_inputs(97, B, T, H, 1, n, p, dt, F32, None, True, F32)
    d["A"] = torch.tensor([-1e10, -1e9])
    d["dt"] = torch.full((B, T, H), 1e-11)
    for t in (20, 21, 64, 127, 140):
        d["dt"][:, t] = 100.0
    w = {k: R.wide(d[k]) for k in ("x", "dt", "A", "B", "C", "D", "h0", "dy", "dhT")}
    e = lambda t: t.expand(-1, -1, H, -1)  # noqa: E731
    x, Bm, C = (w[k].requires_grad_() for k in "xBC")
    ref, hr = R.ssm(x, w["dt"], w["A"], e(Bm), e(C), w["D"], None, w["h0"], None, False)
    ga = torch.autograd.grad((ref * w["dy"]).sum() + (hr * w["dhT"]).sum(), [x, Bm, C])
    xa, Ba, Ca = (w[k].detach().abs().requires_grad_() for k in "xBC")
    ra, ha = R.ssm(xa, w["dt"], w["A"], e(Ba), e(Ca), w["D"].abs(), None, w["h0"].abs(), None, False)
    sa = torch.autograd.grad((ra * w["dy"].abs()).sum() + (ha * w["dhT"].abs()).sum(), [xa, Ba, Ca])
    prod = (2.0 ** -16 if dt == BF else 0.0) + 64 * 2.0 ** -24
    a = [dev(d[k]) for k in ("x", "dt", "A", "B", "C", "D")]
    k = dict(initial_state=dev(d["h0"]), dt_softplus=False, segment_chunks=seg)
    y, h = mixer.ssm_fwd(*a, **k)
    close(y, ref.detach(), ra.detach(), prod, "y")
    close(h, hr.detach(), ha.detach(), 64 * 2.0 ** -24, "state")
    g = mixer.ssm_bwd(*a, None, dev(d["dy"]), d_final_state=dev(d["dhT"]), **k)
    for i, j, what in ((0, 0, "dx"), (3, 1, "dB"), (4, 2, "dC")):
        close(g[i], ga[j], sa[j], 2 * prod, what)

    a[2] = torch.tensor([-float("inf"), -1.0], device="cuda")
    a[1] = torch.full((B, T, H), 0.5, device="cuda")
    y, h = mixer.ssm_fwd(*a, **k)
    x0 = w["x"].detach()[:, :, 0]
    alone = (0.5 * (w["B"] * w["C"]).detach().sum(-1) + w["D"][0]) * x0     # (C delta B + D) x
    size = (0.5 * (w["B"] * w["C"]).detach().abs().sum(-1) + w["D"][0].abs()) * x0.abs()
    close(y[:, :, 0], alone, size, prod, "y without a memory")
    assert bool(torch.isfinite(h).all())


@pytest.mark.parametrize("types", [(BF, F32, F32), (F32, F32, F32)])
def test_ssm_search_of_many_sequences(types):
    """1100 packed sequences: tables of two rounds, searched in two steps."""
    lens = [(0, 1, 2, 0, 0, 1)[i % 6] for i in range(1100)]
    for i, v in ((7, 130), (503, 0), (511, 65), (512, 129), (513, 64), (1023, 66), (1024, 0), (1099, 70)):
        lens[i] = v
    check_ssm(1, sum(lens), 2, 1, 64, 64, tuple(lens), 1, types)


@pytest.mark.parametrize("N,empties", [(1, 0), (63, 3), (64, 70), (65, 5), (130, 200), (4097, 1)])
def test_conv_search_of_sequences(N, empties):
    """Packed sequences of 0 to 5 tokens with runs of empty ones, which the search for a token's
    sequence and the steps from one to the next cross, against the convolution of each alone:
    bit for bit, and the sums of the weights' gradients within fp32 rounding."""
    g = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 6, (N,), generator=g).tolist()
    lens = lens[:N // 2] + [0] * empties + lens[N // 2:] + [3]
    r, D, W = gen(N), 24, 4
    T, M = sum(lens), len(lens)
    x, dy, init, dfin = (dev(t) for t in (r(1, T, D), r(1, T, D), r(M, W - 1, D), r(M, W - 1, D)))
    w, b = dev(r(D, W) * 0.5), dev(r(D) * 0.1)
    cu, host = cu_of(lens)
    k = dict(cu_seqlens=cu, cu_seqlens_host=host)
    y, fin = mixer.conv_fwd(x, w, b, initial_state=init, **k)
    dx, dw, db, di = mixer.conv_bwd(x, w, b, dy, initial_state=init, d_final_state=dfin, **k)
    # each sequence in a row of its own, with zeros behind it that no token before them sees
    L = max(lens)
    at = torch.zeros(M, L, dtype=torch.long)
    real = torch.zeros(M, L, dtype=torch.bool)
    for i, n in enumerate(lens):
        at[i, :n] = int(host[i]) + torch.arange(n)
        real[i, :n] = True
    at, real = dev(at), dev(real)
    rows = lambda t: t[0][at] * real[..., None]  # noqa: E731
    y1, _ = mixer.conv_fwd(rows(x), w, b, initial_state=init)
    assert torch.equal(y[0], y1[real])
    full = torch.cat([init, rows(x)], 1)
    end = dev(torch.tensor(lens))[:, None] + torch.arange(W - 1, device="cuda")
    assert torch.equal(fin, full.gather(1, end[..., None].expand(-1, -1, D)))
    dx1, dw1, db1, di1 = mixer.conv_bwd(rows(x), w, b, rows(dy), initial_state=init)
    # (the final states' gradients come on top: the last tokens', or the start state's)
    extra = torch.zeros(M, L + W - 1, D, device="cuda").scatter_add(1, end[..., None].expand(-1, -1, D), dfin)
    assert torch.equal(dx[0], (dx1 + extra[:, W - 1:])[real]) and torch.equal(di, di1 + extra[:, :W - 1])
    size = (dy[0].abs().sum(0) * 4 * (1 + float(x.abs().max()))).cpu().double()
    close(dw, dw1.cpu().double(), size[:, None].expand(-1, W), 64 * 2.0 ** -24, "dweight")
    close(db, db1.cpu().double(), size, 64 * 2.0 ** -24, "dbias")


def test_graph_of_many_sequences():
    """A captured forward and backward pass over 90 packed sequences, whose tables are made in the
    graph, replayed between eager runs on other inputs of the same lengths."""
    lens = tuple((0, 1, 70, 5, 130)[i % 5] for i in range(90))
    cu, host = cu_of(lens)
    T = sum(lens)
    sets = [{k: dev(v) for k, v in ssm_inputs(s, 1, T, 2, 1, 64, 64, BF, F32, lens, True).items()} for s in (101, 102, 103)]
    d = {k: v.clone() for k, v in sets[0].items()}

    def run():
        a = [d[x] for x in ("x", "dt", "A", "B", "C", "D", "bias")]
        k = dict(initial_state=d["h0"], cu_seqlens=cu, cu_seqlens_host=host)
        return [*mixer.ssm_fwd(*a, **k), *mixer.ssm_bwd(*a, d["dy"], d_final_state=d["dhT"], **k)]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for new in (sets[1], sets[2], sets[0]):
        for k, t in d.items():
            t.copy_(new[k])
        want = [t.clone() for t in run()]
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, captured))
