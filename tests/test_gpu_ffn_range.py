"""The gated feed-forward block far from values of order one: f16 gradients whose dgate
and dup leave f16's range at the scale of dy, elements of dy that are not finite, gates
at either end of the activations, infinite weights. Against the float64 oracle; the bounds are those of
test_gpu_ffn.py but where a test derives its own."""
import numpy as np
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
import test_gpu_ffn as ffn
from gpu_common import torch_mod
from oracle import tokens as ot
from vae_inputs import rng_for

pytestmark = pytest.mark.gpu

U, FLOOR, SUM = ffn.U, ffn.FLOOR, ffn.SUM


def _put(a, t):
    torch = torch_mod()
    x = torch.from_numpy(np.ascontiguousarray(a)).to(ffn._t(t)).cuda()
    return x, ffn._np(x)


def _check_f16_backward(dy, x, wg, wu, wd, saved, act, got, w_type):
    """As test_gpu_ffn's, but for what f16 cuts off dgate and dup: 2^-25 at the scale that brings the largest |dy| to 4..8, or,
    where the largest of them then lies outside 2^-10..65504, at the one that brings that to 2^14..2^15.

    And SUM counts an operand as no less than f16's smallest normal number, 2^-14. The tensor cores bring the products
    of a step to one exponent, the largest by the operands' exponent fields, and cut off what lies 2^-23 below; a subnormal
    operand's field says 2^-14 whatever its value. So what is cut is 2^-23 of max(|a|, 2^-14) max(|b|, 2^-14): of a dy
    mostly subnormal beside a hidden of 367 it is some sixty times 2^-23 |a b|."""
    gate, up, hidden = saved
    m, c = x.shape
    f = wg.shape[0]
    dx, dwg, dwu, dwd, dgate, dup = ot.gated_ffn_backward(dy, x, wg, wu, wd, gate, up, hidden, act)
    a = np.abs
    n = lambda v, scale=1.0: np.where(v != 0, np.maximum(a(v), 2.0 ** -14 / scale), 0)  # noqa: E731
    value, slope = ot.activation(gate, act)
    dh = dy @ wd
    edh = SUM(c) * (n(dy) @ n(wd))
    gain = 2.0 ** (2 - np.floor(np.log2(a(dy).max())))
    top = max(a(dgate).max(), a(dup).max())
    kept = gain if 2.0 ** -10 <= top * gain <= 65504 else 2.0 ** 14 / top
    tiny = 2.0 ** -25 / kept
    u = U["f16"]
    ev, es = 2.0 ** -21 * a(gate), 2.0 ** -20 * (1 + a(gate) * (1 + gate * gate / 4))
    eup = edh * (a(value) + ev) + a(dh) * ev
    eup = eup + (u + 2.0 ** -22) * (a(dup) + eup) + tiny
    egate = a(up) * (edh * (a(slope) + es) + a(dh) * es)
    egate = egate + (u + 2.0 ** -22) * (a(dgate) + egate) + tiny
    ng, nu = n(a(dgate) + egate, kept), n(a(dup) + eup, kept)
    e = egate @ a(wg) + eup @ a(wu) + SUM(2 * f) * (ng @ n(wg) + nu @ n(wu))
    assert a(dx).max() < 6e4  # (the result itself is a number of f16)
    ffn._within(got[0], dx, e + u * (a(dx) + e) + FLOOR["f16"])
    if got[1] is None:
        return top * gain
    for g, ref, e in ((got[1], dwg, egate.T @ a(x) + SUM(m) * (ng.T @ n(x))),
                      (got[2], dwu, eup.T @ a(x) + SUM(m) * (nu.T @ n(x))),
                      (got[3], dwd, SUM(m) * (n(dy).T @ n(hidden)))):
        ffn._within(g, ref, e + U[w_type] * (a(ref) + e) + FLOOR[w_type])
    return top * gain


def _large(kind, m, c, f, act):
    """Operands of f16 and the saved gate, up and hidden; at the scale of dy the largest of dgate and dup is too large or too
    small for f16 (but for "plain")."""
    r = rng_for(3, f"ffn.range.{kind}.{m}.{c}.{f}.{act}")
    x = r.standard_normal((m, c))
    wg, wu = r.standard_normal((f, c)) / np.sqrt(c) / 64, r.standard_normal((f, c)) / np.sqrt(c) / 64
    gate, up = r.standard_normal((m, f)) * 1.5, r.standard_normal((m, f))
    wd, dy = r.standard_normal((c, f)) / np.sqrt(f), r.standard_normal((m, c)) * 2.0 ** -14
    if kind == "constant":  # dgate and hidden are ordinary numbers of f16, dgate at the scale of dy is none
        dy, wd = np.full((m, c), 2.0 ** -14), np.full((c, f), 2.0 ** -6)
        gate, up = np.full((m, f), 8.0), np.full((m, f), 1024.0)
    elif kind == "up":  # gates near 0 beside a few large ups
        gate = gate / 64
        up[r.random((m, f)) < 0.02] = 1e4
        wd = np.abs(wd)
        dy = np.abs(dy)
    elif kind == "down":  # large weights
        wd, dy = wd * 0 + 16.0, np.full((m, c), 2.0 ** -20)
        gate, up = gate * 0 + 6.0, up * 0 + 50.0
    elif kind == "one":  # a single element
        gate[m // 2, f // 2], up[m // 2, f // 2], dy[m // 2] = 100.0, 600.0, 2.0 ** -12
        wd[:, f // 2] = 1.0
    elif kind == "small":
        gate, up, wd = gate * 2.0 ** -12, up * 2.0 ** -12, wd * 2.0 ** -4
    t = {"x": x, "wg": wg, "wu": wu, "wd": wd, "dy": dy, "gate": gate, "up": up}
    dev, host = {}, {}
    for k, v in t.items():
        dev[k], host[k] = _put(v, "f16")
    dev["hidden"], host["hidden"] = _put(np.clip(ot.activation(host["gate"], act)[0] * host["up"], -6e4, 6e4), "f16")
    return dev, host


def _backward(v, act, **kw):
    return vg.gated_ffn_backward(v["dy"], v["x"], v["wg"], v["wu"], v["wd"], (v["gate"], v["up"], v["hidden"]), activation=act, **kw)


@pytest.mark.parametrize("kind", ["constant", "up", "down", "one", "small"])
@pytest.mark.parametrize("m,c,f,act", [(1, 1152, 40, "silu"), (40, 1152, 264, "gelu"), (300, 1160, 136, "gelu_tanh"), (4300, 1152, 72, "silu")])
def test_f16_gradient_whose_parts_leave_the_range_at_the_scale_of_dy(kind, m, c, f, act):
    torch = torch_mod()
    dev, h = _large(kind, m, c, f, act)
    saved = (h["gate"], h["up"], h["hidden"])
    args = (h["dy"], h["x"], h["wg"], h["wu"], h["wd"], saved, act)
    got = _backward(dev, act, grad_dtype=torch.float32)
    top = _check_f16_backward(*args, got, "f32")
    assert top < 7e-4 if kind == "small" else top > 7e4
    one = _backward(dev, act, weight_grads=False)
    assert torch.equal(one[0], got[0])
    assert all(torch.equal(a, b) for a, b in zip(got, _backward(dev, act, grad_dtype=torch.float32)))


def test_f16_gradient_takes_its_scale_anew_in_every_call():
    """One workspace and one graph for operands that pass the range and for ordinary ones, in turn."""
    torch = torch_mod()
    m, c, f, act = 300, 1160, 136, "silu"
    sets = [_large(k, m, c, f, act)[0] for k in ("plain", "up", "plain", "small", "constant", "plain")]
    refs = [_backward(v, act, grad_dtype=torch.float32) for v in sets]
    assert all(torch.isfinite(g).all() for r in refs for g in r)
    ws = torch.full((vg.gated_ffn_backward_workspace_bytes(m, c, f),), 255, dtype=torch.uint8, device="cuda")
    for v, r in zip(sets, refs):
        assert all(torch.equal(a, b) for a, b in zip(_backward(v, act, grad_dtype=torch.float32, workspace=ws), r))
    held = {k: t.clone() for k, t in sets[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _backward(held, act, grad_dtype=torch.float32, workspace=ws)
    for v, r in zip(sets, refs):
        for k, t in held.items():
            t.copy_(v[k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, r))
    vg.sync_status()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("size", [2.0 ** -20, 1.0])
def test_f16_gradient_of_rows_beside_one_that_is_not_finite(bad, size):
    """Whatever stands in one element of dy, the other rows' dx, and the parts of dw_down that it does not enter, are those
    of a call without it, bit for bit."""
    torch = torch_mod()
    case = (300, 72, 264, "f16", "silu")
    (x, x64), (wg, wg64), (wu, wu64), (wd, _) = ffn._case(case)
    saved, _ = ffn._saved(case, x64, wg64, wu64)
    dy = ffn._draw(7, "range.dy", (300, 72), "f16")[0].clamp(-4, 4) * size
    dy[17, 3] = 5.0 * size  # the largest stays where it is
    ref = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, grad_dtype=torch.float32)
    assert all(torch.isfinite(g).all() for g in ref)
    bdy = dy.clone()
    bdy[201, 70] = bad
    got = vg.gated_ffn_backward(bdy, x, wg, wu, wd, saved, grad_dtype=torch.float32)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[201] = False
    assert torch.equal(got[0][keep], ref[0][keep]) and not torch.isfinite(got[0][201]).any()
    cols = torch.ones(72, dtype=torch.bool, device="cuda")
    cols[70] = False
    assert torch.equal(got[3][cols], ref[3][cols]) and not torch.isfinite(got[3][70]).any()
    nothing = vg.gated_ffn_backward(torch.full_like(dy, float("nan")), x, wg, wu, wd, saved)
    assert all(g.isnan().all() for g in nothing)


@pytest.mark.parametrize("m", [5, 300])
def test_gelu_tanh_at_the_ends_of_bf16(m):
    """Far from 0 the activation is g or 0 and its slope 1 or 0: with dhidden = up = 1 and w_gate = 1/16, dx is a
    sixteenth of the slopes' sum, a number of bf16."""
    torch = torch_mod()
    c, f = 8, 16
    ends = np.array([1e14, -1e14, 2e19, -2e19, 3e38, -3e38, 1e12, -1e12])
    gate = ends[rng_for(5, f"ffn.ends.{m}").integers(0, 8, (m, f))]
    gate, g64 = _put(gate, "bf16")
    one = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    slope = (g64 > 0).astype(np.float64)
    got = vg.gated_ffn_backward(one(m, c), one(m, c), one(f, c) / 16, one(f, c) * 0, one(c, f) / 8, (gate, one(m, f), one(m, f)),
                                activation="gelu_tanh", grad_dtype=torch.float32)
    assert np.array_equal(ffn._np(got[0]), np.repeat(slope.sum(1, keepdims=True) / 16, c, 1))
    assert np.array_equal(ffn._np(got[1]), np.repeat(slope.sum(0)[:, None], c, 1))
    # and forward: gate = x w_gate of one channel, up = 1
    x = torch.zeros(m, c, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = gate[:, 0], 1.0
    wg, wu = one(f, c) * 0, one(f, c) * 0
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    hidden = vg.gated_ffn(x, wg, wu, one(c, f) * 0, activation="gelu_tanh", save=True)[1][2]
    assert np.array_equal(ffn._np(hidden), np.repeat((g64 * slope)[:, :1], f, 1))


@pytest.mark.parametrize("t,low,up", [("bf16", -12.0, 1.0), ("f16", -6.5, 2.0 ** 14)])
def test_gelu_keeps_its_digits_far_below_zero(t, low, up):
    """g Phi(g) and its slope within a relative bound. The tail is e^(-g^2/2) times a polynomial that is fitted to 2^-22.5, in
    some ten roundings (of which the last ones count, 2^-21.5) and two approximate instructions (2^-22): less than 2^-20.
    The exponent is off by 2.5 units of 2^-24 of g^2 / 2 at most, and the exponential by as much relative: under 2^-23 g^2.
    The density has the exponential's part of that. Then one rounding to the type; up and dhidden are powers of two."""
    torch = torch_mod()
    m, c, f = 257, 8, 8
    g, g64 = _put(np.linspace(low, 3.0, m), t)
    value, slope = ot.activation(g64, "gelu")
    pdf = np.exp(-0.5 * g64 * g64) / np.sqrt(2 * np.pi)
    ev = (2.0 ** -20 + 2.0 ** -23 * g64 ** 2) * np.abs(value)
    es = (2.0 ** -20 + 2.0 ** -23 * g64 ** 2) * np.abs(value / np.where(g64 == 0, 1, g64)) + (2.0 ** -21 + 2.0 ** -23 * g64 ** 2) * np.abs(g64) * pdf
    zero = lambda *s: torch.zeros(s, dtype=ffn._t(t), device="cuda")  # noqa: E731
    wg, wu = zero(f, c), zero(f, c)
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    for rows in (slice(0, m), slice(0, 20), slice(100, 132)):  # many tokens and few
        x = zero(m, c)
        x[:, 0], x[:, 1] = g, up
        hidden = vg.gated_ffn(x[rows], wg, wu, zero(c, f), activation="gelu", save=True)[1][2]
        ffn._within(hidden[:, 3], (value * up)[rows], up * (ev + U[t] * (np.abs(value) + ev))[rows] + FLOOR[t])
    # dx takes dgate from one channel and dup from another: dhidden = 1, up = 2^4
    dy, wd = zero(m, c), zero(c, f)
    dy[:, 0], wd[0] = 1.0, 1.0
    wg, wu = zero(f, c), zero(f, c)
    wg[0, 0], wu[0, 1] = 1.0, 1.0
    saved = (g[:, None].repeat(1, f), zero(m, f) + 16, zero(m, f))
    dx = vg.gated_ffn_backward(dy, zero(m, c), wg, wu, wd, saved, activation="gelu", weight_grads=False)[0]
    # 2^-22: the sums' and the scale's way through f32. In f16 two roundings: of dgate and dup at four times their size (dy is
    # 1), where the floor is 2^-25 / 4, and of dx; of a subnormal dx they are different ones (-8.606e-8 comes out as
    # -1.19e-7, 1.11 times a single rounding's bound off)
    tol = lambda ref, e: e + (U[t] + 2.0 ** -22) * (np.abs(ref) + e) + FLOOR[t] * 1.25  # noqa: E731
    ffn._within(dx[:, 0], 16 * slope, tol(16 * slope, 16 * es))
    ffn._within(dx[:, 1], value, tol(value, ev))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 20, 40])
def test_infinite_weights_reach_their_outputs_alone(t, m):
    """An infinite element of w_down makes its column of y infinite, with the sign of hidden; of few tokens too, whose second
    part of hidden may be 0 or have the other sign."""
    torch = torch_mod()
    case = (m, 72, 136, t, "silu")
    (x, _), (wg, _), (wu, _), (wd, _) = ffn._case(case)
    y, saved = vg.gated_ffn(x, wg, wu, wd, save=True)
    bad = wd.clone()
    bad[5, 100], bad[70, 3] = float("inf"), float("-inf")
    z = vg.gated_ffn(x, wg, wu, bad)
    keep = torch.ones(72, dtype=torch.bool, device="cuda")
    keep[5] = keep[70] = False
    assert torch.equal(z[:, keep], y[:, keep])
    hidden = saved[2].float()
    assert (hidden[:, 100] != 0).all() and (hidden[:, 3] != 0).all()
    assert torch.equal(z[:, 5].float(), hidden[:, 100] * float("inf")) and torch.equal(z[:, 70].float(), hidden[:, 3] * float("-inf"))


def test_the_largest_number_of_tokens():
    """2^24 tokens: rows at the ends and around the middle as those of a short call, and zeros elsewhere; the weights'
    gradients, sums of the same 160 terms in another order, each within SUM of the terms' absolute values."""
    torch = torch_mod()
    m, c, f = 1 << 24, 8, 16
    places = [0, m // 2 - 20, 9_000_001, m - 40]
    x, dy = (ffn._draw(11, "far." + n, (160, c), "bf16")[0] for n in ("x", "dy"))
    wg, wu, wd = (ffn._draw(11, "far." + n, s, "bf16", 0.3)[0] for n, s in (("g", (f, c)), ("u", (f, c)), ("d", (c, f))))

    def spread(short):
        long = torch.zeros(m, c, dtype=torch.bfloat16, device="cuda")
        for i, at in enumerate(places):
            long[at:at + 40] = short[40 * i:40 * i + 40]
        return long

    gather = lambda t: torch.cat([t[at:at + 40] for at in places])  # noqa: E731
    y, saved = vg.gated_ffn(spread(x), wg, wu, wd, save=True)
    ry, rsaved = vg.gated_ffn(x, wg, wu, wd, save=True)
    assert torch.equal(gather(y), ry) and all(torch.equal(gather(a), b) for a, b in zip(saved, rsaved))
    assert int((y != 0).any(1).sum()) == int((ry != 0).any(1).sum())
    got = vg.gated_ffn_backward(spread(dy), spread(x), wg, wu, wd, saved, grad_dtype=torch.float32)
    ref = vg.gated_ffn_backward(dy, x, wg, wu, wd, rsaved, grad_dtype=torch.float32)
    assert torch.equal(gather(got[0]), ref[0]) and int((got[0] != 0).any(1).sum()) == int((ref[0] != 0).any(1).sum())
    g, u, h = (ffn._np(t) for t in rsaved)
    *_, dgate, dup = ot.gated_ffn_backward(ffn._np(dy), ffn._np(x), ffn._np(wg), ffn._np(wu), ffn._np(wd), g, u, h)
    for a, b, left, right in ((got[1], ref[1], dgate, ffn._np(x)), (got[2], ref[2], dup, ffn._np(x)), (got[3], ref[3], ffn._np(dy), h)):
        assert (np.abs(ffn._np(a) - ffn._np(b)) <= 2 * SUM(160) * (np.abs(left).T @ np.abs(right))).all()


@pytest.mark.parametrize("m", [20, 40])
def test_the_largest_widths(m):
    """16384 channels over 65536 hidden ones, few tokens and many, both ways, against torch in 64 bits on the GPU; the bounds are those of
    test_gpu_ffn.py."""
    torch = torch_mod()
    c, f, u = 16384, 65536, U["bf16"]
    gen = torch.Generator(device="cuda").manual_seed(12)
    draw = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).bfloat16()  # noqa: E731
    x, dy, wg, wu, wd = draw(m, c), draw(m, c), draw(f, c, std=c ** -0.5), draw(f, c, std=c ** -0.5), draw(c, f, std=f ** -0.5)
    y, saved = vg.gated_ffn(x, wg, wu, wd, save=True)
    near = lambda got, ref, e: (got.double() - ref).abs() <= e + u * (ref.abs() + e)  # noqa: E731
    d = lambda t: t.double()  # noqa: E731
    gate, up, eg, eu = d(x) @ d(wg).T, d(x) @ d(wu).T, SUM(c) * (d(x).abs() @ d(wg).abs().T), SUM(c) * (d(x).abs() @ d(wu).abs().T)
    s = torch.sigmoid(gate)
    eh = up.abs() * (1.13 * eg + 2.0 ** -21 * gate.abs()) + ((gate * s).abs() + 1.13 * eg) * eu + 2.0 ** -23 * (gate * s * up).abs()
    assert all(near(a, b, e).all() for a, b, e in zip(saved, (gate, up, gate * s * up), (eg, eu, eh)))
    h = (gate * s * up).abs()
    assert near(y, (gate * s * up) @ d(wd).T, (eh + u * (h + eh) + SUM(f) * h) @ d(wd).abs().T).all()
    got = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved)
    gate, up, hidden = map(d, saved)
    s = torch.sigmoid(gate)
    value, slope = gate * s, s * (1 + gate * (1 - s))
    dh, edh = d(dy) @ d(wd), SUM(c) * (d(dy).abs() @ d(wd).abs())
    dgate, dup = dh * up * slope, dh * value
    es = 2.0 ** -20 * (1 + gate.abs() * (1 + gate * gate / 4))
    eup = edh * (value.abs() + 2.0 ** -21 * gate.abs()) + dh.abs() * 2.0 ** -21 * gate.abs()
    eup = eup + (u + 2.0 ** -22) * (dup.abs() + eup)
    egate = up.abs() * (edh * (slope.abs() + es) + dh.abs() * es)
    egate = egate + (u + 2.0 ** -22) * (dgate.abs() + egate)
    e = egate @ d(wg).abs() + eup @ d(wu).abs() + SUM(2 * f) * ((dgate.abs() + egate) @ d(wg).abs() + (dup.abs() + eup) @ d(wu).abs())
    assert near(got[0], dgate @ d(wg) + dup @ d(wu), e).all()
    for rows in (slice(0, 2048), slice(f // 2 - 300, f // 2 + 300), slice(f - 2048, f)):  # of hidden
        ax, ad = d(x).abs(), d(dy).abs()
        assert near(got[1][rows], dgate[:, rows].T @ d(x), egate[:, rows].T @ ax + SUM(m) * ((dgate.abs() + egate)[:, rows].T @ ax)).all()
        assert near(got[2][rows], dup[:, rows].T @ d(x), eup[:, rows].T @ ax + SUM(m) * ((dup.abs() + eup)[:, rows].T @ ax)).all()
        assert near(got[3][:, rows], d(dy).T @ hidden[:, rows], SUM(m) * (ad.T @ hidden[:, rows].abs())).all()
    vg.sync_status()
