"""GPU parity of the gated feed-forward block and its gradient against the
float64 oracle.

Tolerances are bounds, element by element, from the arithmetic alone:
- a product over K terms in f32: SUM(K) = 2^-23 (K / 16 + 48) of the sum of
  absolute values: one rounding (or truncation, 2^-23) per sixteen terms and sixteen
  within them, and 32 more where partial sums are joined;
- the activation: |act'| <= 1.13 times the error of its argument, and 2^-21 |g| of
  its own; its derivative 2^-20 (1 + |g| (1 + g^2 / 4)), from 1 - s in f32;
- hidden, dgate and dup in 16 bits, and every result in its type: half a step, U of the
  value (in f16 2^-25 absolute: of dgate and dup at the scale that brings the largest
  |dy| to 4..8)."""
import numpy as np
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from gpu_common import torch_mod
from oracle import tokens as ot
from vae_inputs import rng_for

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def SUM(k):
    return 2.0 ** -23 * (k / 16 + 48)


def _t(name):
    torch = torch_mod()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _draw(seed, name, shape, t, std=1.0):
    torch = torch_mod()
    a = rng_for(seed, "ffn." + name).standard_normal(shape) * std
    x = torch.from_numpy(np.ascontiguousarray(a)).to(_t(t)).cuda()
    return x, x.double().cpu().numpy()


def _np(x):
    return x.double().cpu().numpy()


def _within(got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape
    assert not np.isnan(got).any()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


# m, c, f, type, activation
CASES = [(1, 8, 8, "bf16", "silu"), (1, 64, 64, "f16", "gelu"), (3, 16, 40, "bf16", "gelu_tanh"), (8, 1152, 4608, "bf16", "silu"),
         (17, 264, 520, "f16", "silu"), (33, 72, 136, "bf16", "gelu"), (64, 1288, 2056, "f16", "gelu_tanh"),
         (127, 72, 136, "f16", "silu"), (128, 64, 128, "bf16", "silu"), (129, 128, 256, "f16", "gelu"),
         (255, 200, 264, "bf16", "gelu"), (257, 136, 512, "bf16", "silu"), (256, 512, 2048, "f16", "silu"),
         (300, 576, 1000, "bf16", "gelu_tanh"), (513, 1152, 328, "f16", "silu"), (1000, 264, 520, "bf16", "silu"),
         (5000, 64, 1024, "f16", "gelu"), (20000, 64, 72, "bf16", "silu"), (3000, 520, 2048, "bf16", "silu"),
         (70000, 8, 24, "f16", "gelu_tanh"),
         # few tokens: one piece of the contraction and many, rows that end inside a block, contractions over a cluster
         (2, 8, 4608, "f16", "gelu"), (16, 1152, 1160, "f16", "gelu"), (32, 2304, 72, "bf16", "gelu_tanh"), (31, 24, 6008, "bf16", "silu"),
         (9, 328, 40, "f16", "silu"), (33, 2304, 2056, "bf16", "silu"),
         # tiles of 512 rows, the last ones half and hardly filled; long sums over few tiles beside short ones over many
         (4100, 576, 2304, "f16", "gelu"), (4353, 640, 2568, "bf16", "silu"), (41001, 72, 136, "bf16", "gelu_tanh")]


def _case(case):
    m, c, f, t, act = case
    x = _draw(1, f"x.{case}", (m, c), t)
    wg = _draw(1, f"wg.{case}", (f, c), t, 1.5 / np.sqrt(c))
    wu = _draw(1, f"wu.{case}", (f, c), t, 1.0 / np.sqrt(c))
    wd = _draw(1, f"wd.{case}", (c, f), t, 1.0 / np.sqrt(f))
    return x, wg, wu, wd


def _forward_bounds(case, x, wg, wu, wd, gate, up, hidden):
    """How far (gate, up, hidden, y in f32) may be off before their own rounding to the type; hidden's included in y."""
    m, c, f, t, act = case
    eg, eu = SUM(c) * (np.abs(x) @ np.abs(wg).T), SUM(c) * (np.abs(x) @ np.abs(wu).T)
    value = np.abs(ot.activation(gate, act)[0])
    eh = np.abs(up) * (1.13 * eg + 2.0 ** -21 * np.abs(gate)) + (value + 1.13 * eg) * eu + 2.0 ** -23 * np.abs(hidden)
    ey = (eh + U[t] * (np.abs(hidden) + eh) + FLOOR[t]) @ np.abs(wd).T + SUM(f) * (np.abs(hidden) @ np.abs(wd).T)
    return eg, eu, eh, ey


def _check_forward(case, x, wg, wu, wd, y, saved, y_type, residual=0.0):
    t = case[3]
    ry, gate, up, hidden = ot.gated_ffn(x, wg, wu, wd, case[4])
    eg, eu, eh, ey = _forward_bounds(case, x, wg, wu, wd, gate, up, hidden)
    if saved is not None:
        for got, ref, e in zip(saved, (gate, up, hidden), (eg, eu, eh)):
            _within(got, ref, e + U[t] * (np.abs(ref) + e) + FLOOR[t])
    ref = ry + residual
    _within(y, ref, ey + U[y_type] * (np.abs(ref) + ey) + FLOOR[y_type])


@pytest.mark.parametrize("case", CASES)
def test_gated_ffn(case):
    torch = torch_mod()
    m, c, f, t, act = case
    (x, x64), (wg, wg64), (wu, wu64), (wd, wd64) = _case(case)
    out = torch.full((m, c), float("nan"), dtype=_t(t), device="cuda")
    y = vg.gated_ffn(x, wg, wu, wd, activation=act, out=out)
    assert y is out
    _check_forward(case, x64, wg64, wu64, wd64, y, None, t)
    y2, saved = vg.gated_ffn(x, wg, wu, wd, activation=act, save=True)
    _check_forward(case, x64, wg64, wu64, wd64, y2, saved, t)
    assert torch.equal(vg.gated_ffn(x, wg, wu, wd, activation=act), y)
    # the f32 stream, alone and added in place
    y3 = vg.gated_ffn(x, wg, wu, wd, activation=act, out_dtype=torch.float32)
    _check_forward(case, x64, wg64, wu64, wd64, y3, None, "f32")
    r, r64 = _draw(2, f"res.{case}", (m, c), "f32")
    assert vg.gated_ffn(x, wg, wu, wd, activation=act, residual=r, out=r) is r
    _check_forward(case, x64, wg64, wu64, wd64, r, None, "f32", r64)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] <= 32])
def test_few_tokens_keep_what_the_rounding_of_hidden_left(case):
    """Up to 32 tokens the second product takes hidden in two parts. The second part is rounded too: U^2 of hidden, in f16
    (where it is held times 2^11) at least 2^-36. Both parts' sums are joined by one more rounding each."""
    torch = torch_mod()
    m, c, f, t, act = case
    (x, x64), (wg, wg64), (wu, wu64), (wd, wd64) = _case(case)
    ref, gate, up, hidden = ot.gated_ffn(x64, wg64, wu64, wd64, act)
    _, _, eh, _ = _forward_bounds(case, x64, wg64, wu64, wd64, gate, up, hidden)
    a = np.abs
    e = (eh + U[t] ** 2 * (a(hidden) + eh) + FLOOR[t] / 2048) @ a(wd64).T + SUM(f) * ((1 + 2 * U[t]) * (a(hidden) + eh) @ a(wd64).T)
    _within(vg.gated_ffn(x, wg, wu, wd, activation=act, out_dtype=torch.float32), ref, e + 2.0 ** -22 * (a(ref) + e))
    y, _ = vg.gated_ffn(x, wg, wu, wd, activation=act, save=True)
    assert torch.equal(y, vg.gated_ffn(x, wg, wu, wd, activation=act))
    _within(y, ref, e + U[t] * (a(ref) + e) + FLOOR[t] + 2.0 ** -22 * a(ref))


def test_few_tokens_whose_hidden_passes_f16():
    torch = torch_mod()
    x = torch.ones(2, 8, dtype=torch.float16, device="cuda")
    wg, wu = torch.full((16, 8), 64.0, dtype=torch.float16, device="cuda"), torch.full((16, 8), 64.0, dtype=torch.float16, device="cuda")
    wd = torch.full((8, 16), 2.0 ** -10, dtype=torch.float16, device="cuda")
    y, saved = vg.gated_ffn(x, wg, wu, wd, save=True, out_dtype=torch.float32)
    assert torch.isinf(saved[2]).all() and torch.isinf(y).all()  # 512 * 512 is no f16: infinite, and no NaN from its rest


def _check_backward(case, dy, x, wg, wu, wd, gate, up, hidden, got, w_type):
    m, c, f, t, act = case
    dx, dwg, dwu, dwd, dgate, dup = ot.gated_ffn_backward(dy, x, wg, wu, wd, gate, up, hidden, act)
    value, slope = ot.activation(gate, act)
    dh = dy @ wd
    edh = SUM(c) * (np.abs(dy) @ np.abs(wd))
    tiny = FLOOR[t] * max(np.abs(dy).max(), 2.0 ** -24) / 4
    ev, es = 2.0 ** -21 * np.abs(gate), 2.0 ** -20 * (1 + np.abs(gate) * (1 + gate * gate / 4))
    eup = edh * (np.abs(value) + ev) + np.abs(dh) * ev
    eup = eup + (U[t] + 2.0 ** -22) * (np.abs(dup) + eup) + tiny
    egate = np.abs(up) * (edh * (np.abs(slope) + es) + np.abs(dh) * es)
    egate = egate + (U[t] + 2.0 ** -22) * (np.abs(dgate) + egate) + tiny
    a = np.abs
    e = egate @ a(wg) + eup @ a(wu) + SUM(2 * f) * ((a(dgate) + egate) @ a(wg) + (a(dup) + eup) @ a(wu))
    _within(got[0], dx, e + U[t] * (a(dx) + e) + FLOOR[t])
    if got[1] is None:
        return
    for g, ref, e in ((got[1], dwg, egate.T @ a(x) + SUM(m) * ((a(dgate) + egate).T @ a(x))),
                      (got[2], dwu, eup.T @ a(x) + SUM(m) * ((a(dup) + eup).T @ a(x))),
                      (got[3], dwd, SUM(m) * (a(dy).T @ a(hidden)))):
        _within(g, ref, e + U[w_type] * (a(ref) + e) + FLOOR[w_type])


def _saved(case, x, wg, wu):
    """gate, up and hidden in the type, as a forward pass leaves them."""
    torch = torch_mod()
    t = _t(case[3])
    gate, up = x @ wg.T, x @ wu.T
    hidden = ot.activation(gate, case[4])[0] * up
    s = tuple(torch.from_numpy(a).to(t).cuda() for a in (gate, up, hidden))
    return s, tuple(_np(a) for a in s)


@pytest.mark.parametrize("case", CASES)
def test_gated_ffn_backward(case):
    torch = torch_mod()
    m, c, f, t, act = case
    (x, x64), (wg, wg64), (wu, wu64), (wd, wd64) = _case(case)
    saved, s64 = _saved(case, x64, wg64, wu64)
    dy, dy64 = _draw(3, f"dy.{case}", (m, c), t)
    nan = lambda *s, t=t: torch.full(s, float("nan"), dtype=_t(t), device="cuda")  # noqa: E731
    got = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, activation=act, dx=nan(m, c), dw_gate=nan(f, c), dw_up=nan(f, c),
                                dw_down=nan(c, f))
    _check_backward(case, dy64, x64, wg64, wu64, wd64, *s64, got, t)
    again = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, activation=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    one = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, activation=act, weight_grads=False)
    assert torch.equal(one[0], got[0]) and one[1:] == (None, None, None)
    got = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, activation=act, grad_dtype=torch.float32)
    _check_backward(case, dy64, x64, wg64, wu64, wd64, *s64, got, "f32")


@pytest.mark.parametrize("gain", [2.0 ** -20, 2.0 ** -10, 1.0, 2.0 ** 10])
def test_gated_ffn_backward_f16_gradients_of_any_size(gain):
    """dgate and dup keep their digits whatever the size of dy: the weights' gradients in f32 are the same times the
    gain, bit for bit, where dy's values are normal numbers times it. (2^-20 brings them below 2^-14. What the tensor
    cores cut off a sum is counted from the operands' exponents, and subnormal ones have the lowest exponent whatever
    their value, so other bits may go: up to 2^-23 of the absolute values per sixteen terms on either side, which is
    what SUM counts. There the results are held to the bound against float64, as everywhere.)"""
    torch = torch_mod()
    case = (200, 72, 136, "f16", "silu")
    (x, x64), (wg, wg64), (wu, wu64), (wd, wd64) = _case(case)
    saved, s64 = _saved(case, x64, wg64, wu64)
    dy = (torch.from_numpy(rng_for(4, "ffn.any").integers(-8, 9, (200, 72))).cuda().half() / 4)
    ref = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, grad_dtype=torch.float32)
    got = vg.gated_ffn_backward(dy * gain, x, wg, wu, wd, saved, grad_dtype=torch.float32)
    _check_backward(case, _np(dy * gain), x64, wg64, wu64, wd64, *s64, got, "f32")
    if gain >= 2.0 ** -10:
        assert all(torch.equal(a / gain, b) for a, b in zip(got[1:], ref[1:]))
    zero = vg.gated_ffn_backward(torch.zeros_like(dy), x, wg, wu, wd, saved)
    assert all((a == 0).all() for a in zero)


def test_gated_ffn_backward_against_differences():
    """The whole gradient against differences of the forward in its f32 output. Both sides round hidden, dgate and dup
    (2^-8 each) and the differences divide the output's errors by the step: 2^-6 of the sum of absolute values, and
    the third derivatives' h^2."""
    torch = torch_mod()
    case = (6, 16, 24, "bf16", "gelu_tanh")
    (x, _), (wg, _), (wu, _), (wd, _) = _case(case)
    wy = _draw(5, "wy", (6, 16), "bf16")[0]
    _, saved = vg.gated_ffn(x, wg, wu, wd, activation="gelu_tanh", save=True)
    grads = vg.gated_ffn_backward(wy, x, wg, wu, wd, saved, activation="gelu_tanh", grad_dtype=torch.float32)

    def loss(*a):
        return (vg.gated_ffn(*a, activation="gelu_tanh", out_dtype=torch.float32) * wy).double().sum().item()

    size = (vg.gated_ffn(x, wg, wu, wd, activation="gelu_tanh", out_dtype=torch.float32).abs() * wy.abs()).double().sum().item()
    h = 0.25
    for i, g in enumerate(grads):
        args = [x, wg, wu, wd]
        v = torch.sign(_draw(6, f"v{i}", args[i].shape, "f32")[0])
        # steps that 16 bits hold: the difference of the two rounded points, in f32
        up, down = list(args), list(args)
        up[i], down[i] = (args[i].float() + h * v * args[i].float().abs()).bfloat16(), (args[i].float() - h * v * args[i].float().abs()).bfloat16()
        num = loss(*up) - loss(*down)
        ref = (g.float() * (up[i].float() - down[i].float())).double().sum().item()
        whole = (g.float().abs() * (up[i].float() - down[i].float()).abs()).double().sum().item()
        assert abs(num - ref) <= 2.0 ** -6 * (whole + size) + h * h * whole, (i, num, ref, whole, size)


def test_gated_ffn_values_that_are_not_finite_stay_in_their_rows():
    torch = torch_mod()
    case = (300, 72, 264, "bf16", "silu")
    (x, x64), (wg, wg64), (wu, wu64), (wd, _) = _case(case)
    y = vg.gated_ffn(x, wg, wu, wd)
    saved, _ = _saved(case, x64, wg64, wu64)
    dy = _draw(7, "nan.dy", (300, 72), "bf16")[0]
    dx = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved)[0]
    bad = x.clone()
    bad[299, 5] = float("nan")
    bad[7, 71] = float("inf")
    z = vg.gated_ffn(bad, wg, wu, wd)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[299] = keep[7] = False
    assert torch.equal(z[keep], y[keep]) and z[299].isnan().all() and not torch.isfinite(z[7]).any()
    bdy = dy.clone()
    bdy[0, 0] = float("nan")
    got = vg.gated_ffn_backward(bdy, x, wg, wu, wd, saved)
    assert torch.equal(got[0][1:], dx[1:]) and got[0][0].isnan().all() and got[3][0].isnan().all() and torch.isfinite(got[3][1:]).all()


def test_gated_ffn_memory_around_is_left_alone():
    """Results that end inside tiles, in the middle of larger buffers."""
    torch = torch_mod()
    case = (130, 72, 136, "bf16", "gelu")
    m, c, f = case[:3]
    (x, x64), (wg, wg64), (wu, wu64), (wd, _) = _case(case)
    saved, _ = _saved(case, x64, wg64, wu64)
    pad = 512

    def inside(rows, cols, dtype=torch.bfloat16):
        buf = torch.full((rows * cols + 2 * pad,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[pad:pad + rows * cols].view(rows, cols)

    y, dx, dg, du, dd = inside(m, c), inside(m, c), inside(f, c), inside(f, c), inside(c, f)
    ws = torch.full((vg.gated_ffn_workspace_bytes(m, c, f) + 1024,), 9, dtype=torch.uint8, device="cuda")
    vg.gated_ffn(x, wg, wu, wd, activation="gelu", out=y[1], workspace=ws[:-1024])
    wb = torch.full((vg.gated_ffn_backward_workspace_bytes(m, c, f) + 1024,), 9, dtype=torch.uint8, device="cuda")
    vg.gated_ffn_backward(y[1].contiguous().clone(), x, wg, wu, wd, saved, activation="gelu", dx=dx[1], dw_gate=dg[1], dw_up=du[1],
                          dw_down=dd[1], workspace=wb[:-1024])
    for buf, _ in (y, dx, dg, du, dd):
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
    assert (ws[-1024:] == 9).all() and (wb[-1024:] == 9).all()
    r = inside(m, c, torch.float32)
    vg.gated_ffn(x, wg, wu, wd, activation="gelu", residual=torch.zeros(m, c, device="cuda"), out=r[1])
    assert (r[0][:pad] == 7).all() and (r[0][-pad:] == 7).all()


@pytest.mark.parametrize("m", [1, 24, 300])
def test_gated_ffn_streams_graphs_and_halves_of_one_weight(m):
    torch = torch_mod()
    case = (m, 136, 264, "f16", "silu")
    (x, x64), (wg, wg64), (wu, wu64), (wd, _) = _case(case)
    saved, _ = _saved(case, x64, wg64, wu64)
    dy = _draw(8, "st.dy", (m, 136), "f16")[0]
    ref = (vg.gated_ffn(x, wg, wu, wd), *vg.gated_ffn_backward(dy, x, wg, wu, wd, saved))
    both = torch.cat((wg, wu))
    assert torch.equal(vg.gated_ffn(x, both[:264], both[264:], wd), ref[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (vg.gated_ffn(x, wg, wu, wd, stream=side), *vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # two graphs on one workspace, replayed in turn, their inputs changed between
    ws = torch.empty(max(vg.gated_ffn_workspace_bytes(m, 136, 264), vg.gated_ffn_backward_workspace_bytes(m, 136, 264)),
                     dtype=torch.uint8, device="cuda")
    xin, dyin = x.clone(), dy.clone()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        ya = vg.gated_ffn(xin, wg, wu, wd, workspace=ws)
    with torch.cuda.graph(gb):
        yb = vg.gated_ffn_backward(dyin, xin, wg, wu, wd, saved, workspace=ws)
    for k in (2.0, 1.0):
        xin.copy_(x * k)
        dyin.copy_(dy * k)
        ga.replay()
        gb.replay()
        ga.replay()
    torch.cuda.synchronize()
    assert torch.equal(ya, ref[0]) and all(torch.equal(a, b) for a, b in zip(yb, ref[1:]))
    vg.sync_status()


def test_gated_ffn_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows are as those of a short call."""
    torch = torch_mod()
    m, c, f = (1 << 18) + 40, 8, 8200
    x = torch.zeros(m, c, dtype=torch.bfloat16, device="cuda")
    tail, _ = _draw(9, "big.x", (40, c), "bf16")
    x[-40:] = tail
    wg, wu, wd = (_draw(9, "big." + n, s, "bf16", 0.2)[0] for n, s in (("g", (f, c)), ("u", (f, c)), ("d", (c, f))))
    y, saved = vg.gated_ffn(x, wg, wu, wd, save=True)
    small, s2 = vg.gated_ffn(tail, wg, wu, wd, save=True)
    near = lambda a, b: (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()  # noqa: E731
    assert near(y[-40:], small) and all(near(a[-40:], b) for a, b in zip(saved, s2)) and (y[:1000] == 0).all()
    dy = torch.zeros_like(x)
    dy[-40:] = small
    got = vg.gated_ffn_backward(dy, x, wg, wu, wd, saved, grad_dtype=torch.float32)
    ref = vg.gated_ffn_backward(small, tail, wg, wu, wd, s2, grad_dtype=torch.float32)
    assert near(got[0][-40:], ref[0]) and all(near(a, b) for a, b in zip(got[1:], ref[1:]))
