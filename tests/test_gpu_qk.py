"""GPU parity of the norm of query and key heads with rotary positions, and of
its gradient, against the float64 oracle.

Tolerances are bounds, element by element, from the arithmetic alone: the
rounding of the result (half a step, U of its value; 2^-25 absolute in f16); the
root of the mean square over at most 256 channels, chains of at most 16 roundings
of 2^-24 and a 2-ulp rsqrt, halved by the root: 2^-20; the products behind it, two
roundings; the angle, a few 2^-24 turns, and the turn: 2^-20 of |a| + |b| of the
pair, as for rope. Together 2^-19 of the pair. dgamma adds SUM = 2^-17 of the sum
of absolute values (128 roundings along its longest chain, twice over)."""
import numpy as np
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from gpu_common import torch_mod
from oracle import tokens as ot
from vae_inputs import rng_for

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
SUM = 2.0 ** -17
EPS = 1e-5


def _t(name):
    torch = torch_mod()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _draw(seed, name, shape, t, std=1.0, mean=0.0):
    torch = torch_mod()
    a = rng_for(seed, "qk." + name).standard_normal(shape) * std + mean
    x = torch.from_numpy(np.ascontiguousarray(a)).to(_t(t)).cuda()
    return x, x.double().cpu().numpy()


def _np(x):
    return x.double().cpu().numpy()


def _within(got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape
    assert not np.isnan(got).any()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


def _pair_sum(z, rot, inter):
    """|a| + |b| of each element's pair, |z| of the channels that do not turn."""
    p = np.abs(z).copy()
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    p[..., ia] = p[..., ib] = np.abs(z[..., ia]) + np.abs(z[..., ib])
    return p


# b, s, hq, hk, d, axes (None: no positions), type, interleaved, int positions, per batch, gammas
CASES = [(1, 1, 1, 1, 1, None, "f32", True, True, False, True), (2, 3, 2, 1, 2, (2,), "f16", True, False, False, False),
         (2, 5, 3, 2, 10, (2, 6), "f16", False, False, True, True), (1, 256, 8, 8, 64, (32, 32), "bf16", True, True, False, True),
         (8, 1, 16, 4, 128, (0, 64, 64), "bf16", False, False, True, True), (2, 33, 6, 2, 128, (16, 56, 56), "f16", True, False, True, True),
         (1, 700, 5, 5, 96, (0, 32, 32), "f16", False, True, True, True), (3, 19, 2, 1, 256, (64, 64, 64, 64), "f32", True, False, True, True),
         (1, 50, 4, 3, 72, (8, 24, 24), "f32", False, True, False, False), (2, 41, 7, 1, 72, (4, 16, 16), "bf16", True, False, True, True),
         (1, 50, 4, 2, 66, (2, 32, 32), "f16", True, True, False, True), (2, 1000, 20, 5, 40, (8, 16, 16), "bf16", False, False, True, True),
         (1, 333, 3, 3, 40, (4, 8, 8), "f16", False, False, False, True), (1, 9, 2, 2, 256, (2,), "f16", True, True, False, True),
         (1, 700, 3, 1, 255, (2,), "bf16", False, False, False, True), (2, 5, 2, 2, 253, (100, 2, 0, 8), "f32", False, True, True, True),
         (1, 37, 1, 1, 8, (8,), "bf16", False, False, False, True), (1, 37, 1, 1, 16, (16,), "f16", False, False, False, True),
         (1, 37, 2, 3, 24, (8,), "f32", False, False, False, True), (3, 1500, 4, 2, 80, (0, 40, 40), "f32", False, False, True, True),
         (3, 1500, 4, 2, 80, (0, 20, 20), "bf16", False, False, True, True), (2, 100, 3, 2, 64, None, "bf16", True, False, False, True),
         (2, 100, 3, 2, 120, None, "f16", False, False, False, False), (1, 2600, 9, 9, 128, (16, 56, 56), "bf16", False, True, True, True),
         # enough tokens for the gradient's longest turns, the last one short, each way of lying over lanes
         (2, 2601, 5, 2, 64, (0, 32, 32), "bf16", False, True, True, True), (1, 5003, 3, 1, 72, (8, 24, 24), "f16", False, False, False, True),
         (1, 5003, 2, 3, 96, (8, 24, 24), "f16", True, False, False, True), (1, 10007, 1, 1, 256, (128, 64, 64), "bf16", True, True, False, True)]


def _case(case):
    torch = torch_mod()
    b, s, hq, hk, d, axes, t, inter, ints, per, gammas = case
    q, q64 = _draw(1, f"q.{case}", (b, s, hq, d), t, 1.7, 0.2)
    k, k64 = _draw(1, f"k.{case}", (b, s, hk, d), t, 0.4)
    gq, gq64 = _draw(1, f"gq.{case}", (d,), "f32", 0.3, 1.0) if gammas else (None, None)
    gk, gk64 = _draw(1, f"gk.{case}", (d,), "f32", 0.3, 1.0) if gammas else (None, None)
    p = pos = plan = None
    if axes is not None:
        pos = rng_for(1, f"qk.pos.{case}").integers(0, 1500, ((b, s) if per else (s,)) + (len(axes),))
        pos = pos if ints else pos + 0.25
        p = torch.from_numpy(np.asarray(pos, np.int32 if ints else np.float32)).cuda()
        plan = vg.RopePlan(axes, theta=10000.0, interleaved=inter)
    return q, q64, k, k64, gq, gq64, gk, gk64, p, pos, plan


def _check_forward(out, x64, g64, pos, axes, inter, t):
    ref = ot.qk_norm_rope(x64, g64, pos, axes or (), 10000.0, inter, EPS)
    z = ot.qk_norm_rope(x64, g64, eps=EPS)
    _within(out, ref, U[t] * np.abs(ref) * 1.001 + FLOOR[t] + 2.0 ** -19 * _pair_sum(z, sum(axes or ()), inter))


@pytest.mark.parametrize("case", CASES)
def test_qk_norm_rope(case):
    torch = torch_mod()
    axes, t, inter = case[5], case[6], case[7]
    q, q64, k, k64, gq, gq64, gk, gk64, p, pos, plan = _case(case)
    nan = lambda x: torch.full_like(x, float("nan"))  # noqa: E731
    qo, ko = vg.qk_norm_rope(q, k, gq, gk, p, plan, eps=EPS, q_out=nan(q), k_out=nan(k))
    _check_forward(qo, q64, gq64, pos, axes, inter, t)
    _check_forward(ko, k64, gk64, pos, axes, inter, t)
    new = vg.qk_norm_rope(q, k, gq, gk, p, plan, eps=EPS)
    assert torch.equal(new[0], qo) and torch.equal(new[1], ko)
    a, c = q.clone(), k.clone()
    got = vg.qk_norm_rope(a, c, gq, gk, p, plan, eps=EPS, q_out=a, k_out=c)
    assert got[0] is a and got[1] is c and torch.equal(a, qo) and torch.equal(c, ko)


def _check_backward(dx, dg, dy64, x64, g64, pos, axes, inter, t):
    rx, rg = ot.qk_norm_rope_backward(dy64, x64, g64, pos, axes or (), 10000.0, inter, EPS)
    g = np.ones(x64.shape[-1]) if g64 is None else np.abs(g64)
    u = dy64 if pos is None else ot.rope(dy64, pos, axes, 10000.0, inter, inverse=True)
    size = np.sqrt((x64 * x64).mean(-1, keepdims=True) + EPS)
    n = np.abs(x64 / size)
    eu = 2.0 ** -20 * _pair_sum(dy64, sum(axes or ()), inter)
    v, ev = np.abs(u) * g, g * (eu + 2.0 ** -23 * np.abs(u))
    mean = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    along = mean(v * n)
    ealong = mean(ev * n) + 2.0 ** -19 * along
    tol = U[t] * np.abs(rx) * 1.001 + FLOOR[t] + 1.01 * (ev + n * ealong + 2.0 ** -20 * (v + n * along)) / size
    _within(dx, rx, tol)
    if dg is not None:
        un = np.abs(u) * n
        _within(dg, rg, (eu * n + 2.0 ** -20 * un + SUM * un).sum((0, 1, 2)) + U["f32"] * np.abs(rg))


@pytest.mark.parametrize("case", CASES)
def test_qk_norm_rope_backward(case):
    torch = torch_mod()
    d, axes, t, inter = case[4:8]
    q, q64, k, k64, gq, gq64, gk, gk64, p, pos, plan = _case(case)
    dyq, dyq64 = _draw(2, f"dq.{case}", q64.shape, t)
    dyk, dyk64 = _draw(2, f"dk.{case}", k64.shape, t)
    nan = lambda x: torch.full_like(x, float("nan"))  # noqa: E731
    f = lambda: torch.full((d,), float("nan"), device="cuda")  # noqa: E731
    dq, dk, dgq, dgk = vg.qk_norm_rope_backward(dyq, dyk, q, k, gq, gk, p, plan, eps=EPS, dq=nan(q), dk=nan(k),
                                                dgamma_q=f(), dgamma_k=f())
    _check_backward(dq, dgq, dyq64, q64, gq64, pos, axes, inter, t)
    _check_backward(dk, dgk, dyk64, k64, gk64, pos, axes, inter, t)
    again = vg.qk_norm_rope_backward(dyq, dyk, q, k, gq, gk, p, plan, eps=EPS)
    assert all(torch.equal(a, c) for a, c in zip(again, (dq, dk, dgq, dgk)))
    # in place of the gradients, or of the inputs; without the weights' gradients
    a, c = dyq.clone(), k.clone()
    got = vg.qk_norm_rope_backward(a, dyk, q, c, gq, gk, p, plan, eps=EPS, weight_grads=False, dq=a, dk=c)
    assert got[0] is a and got[1] is c and got[2] is None and torch.equal(a, dq) and torch.equal(c, dk)


def test_qk_norm_rope_backward_against_differences():
    """The gradient's direction against differences of the forward, all in f32: steps of 2^-7 give (1e-2)^2 of
    third derivatives of order one; 1e-2 of the whole."""
    torch = torch_mod()
    case = (1, 6, 3, 2, 24, (4, 8, 8), "f32", True, True, False, True)
    q, _, k, _, gq, _, gk, _, p, _, plan = _case(case)
    wq, wk = _draw(3, "wq", q.shape, "f32")[0], _draw(3, "wk", k.shape, "f32")[0]
    dq, dk, dgq, dgk = vg.qk_norm_rope_backward(wq, wk, q, k, gq, gk, p, plan, eps=EPS)

    def loss(q, k, gq, gk):
        a, b = vg.qk_norm_rope(q, k, gq, gk, p, plan, eps=EPS)
        return ((a * wq).double().sum() + (b * wk).double().sum()).item()

    h = 2.0 ** -7
    for i, (x, g) in enumerate(((q, dq), (k, dk), (gq, dgq), (gk, dgk))):
        v = _draw(4, f"v{i}", x.shape, "f32")[0]
        up, down = [q, k, gq, gk], [q, k, gq, gk]
        up[i], down[i] = x + h * v, x - h * v
        num = (loss(*up) - loss(*down)) / (2 * h)
        ref = (g * v).double().sum().item()
        assert abs(num - ref) <= 1e-2 * (g.abs() * v.abs()).double().sum().item()


def test_qk_norm_rope_views_and_caches():
    """Parts of a joint projection in, the keys straight into their rows of a cache; what lies around stays."""
    torch = torch_mod()
    b, s, hq, hk, d = 2, 45, 6, 2, 64
    for off in (0, 1):  # (rows off the 16-byte boundaries too)
        rows = _draw(5, f"joint{off}", (b, s, (hq + 2 * hk) * d + 8 + off), "bf16")[0]
        joint = rows[..., off:off + (hq + 2 * hk) * d].unflatten(-1, (hq + 2 * hk, d))
        q, k = joint[:, :, :hq], joint[:, :, hq:hq + hk]
        pos = torch.arange(s, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2).contiguous()
        plan = vg.RopePlan((32, 32), interleaved=off == 0)
        gq, gk = _draw(5, "gq", (d,), "f32", 0.2, 1.0)[0], _draw(5, "gk", (d,), "f32", 0.2, 1.0)[0]
        ref = vg.qk_norm_rope(q.contiguous(), k.contiguous(), gq, gk, pos, plan)
        cache = torch.full((b, 100, hk, d), 7.0, dtype=torch.bfloat16, device="cuda")
        got = vg.qk_norm_rope(q, k, gq, gk, pos, plan, k_out=cache[:, 30:30 + s])
        near = lambda a, c: (a.float() - c.float()).abs().max() <= 2.0 ** -7 * c.float().abs().max()  # noqa: E731
        assert near(got[0], ref[0]) and near(cache[:, 30:30 + s], ref[1])
        assert (cache[:, :30] == 7).all() and (cache[:, 30 + s:] == 7).all()
        keep = rows.clone()
        dq, dk = _draw(5, "dq", q.shape, "bf16")[0], _draw(5, "dk", k.shape, "bf16")[0]
        want = vg.qk_norm_rope_backward(dq, dk, q.contiguous(), k.contiguous(), gq, gk, pos, plan)
        # the gradients into the parts of a joint gradient, heads before tokens in dq_out
        dj = torch.full((b, s, hq + 2 * hk, d), 5.0, dtype=torch.bfloat16, device="cuda")
        res = vg.qk_norm_rope_backward(dq.transpose(1, 2).contiguous().transpose(1, 2), dk, q, k, gq, gk, pos, plan,
                                       dq=dj[:, :, :hq], dk=dj[:, :, hq:hq + hk])
        assert near(dj[:, :, :hq], want[0]) and near(dj[:, :, hq:hq + hk], want[1]) and (dj[:, :, hq + hk:] == 5).all()
        assert all((a - c).abs().max() <= SUM * 45 * 2 * 6 * 16 for a, c in zip(res[2:], want[2:]))
        assert torch.equal(rows, keep)
        # broadcast inputs: one head read as several
        one = vg.qk_norm_rope(q[:, :, :1].expand(b, s, 3, d), k, gq, gk, pos, plan)[0]
        assert torch.equal(one[:, :, 0], one[:, :, 2]) and near(one[:, :, 0], ref[0][:, :, 0])


def test_qk_norm_rope_zero_rows_and_values_that_are_not_finite():
    torch = torch_mod()
    for d, t in ((64, torch.bfloat16), (33, torch.float32)):
        q = torch.randn(1, 4, 2, d, device="cuda").to(t)
        k = q.clone()
        clean = vg.qk_norm_rope(q, k)[0].clone()
        q[0, 1, 0] = 0
        q[0, 2, 1, 5] = float("nan")
        qo, ko = vg.qk_norm_rope(q, k)
        assert (qo[0, 1, 0] == 0).all() and qo[0, 2, 1].isnan().all()
        rest = torch.ones(1, 4, 2, dtype=torch.bool, device="cuda")
        rest[0, 1, 0] = rest[0, 2, 1] = False
        assert torch.equal(qo[rest], clean[rest]) and torch.equal(ko, clean)
        q[0, 2, 1, 5] = 1.0
        dq, _, dgq, _ = vg.qk_norm_rope_backward(torch.ones_like(q), torch.ones_like(k), q, k, eps=1e-6)
        assert torch.isfinite(dq[0, 0]).all() and torch.isfinite(dgq).all()
        # a zero row's gradient is dy / sqrt(eps)
        want = torch.full((d,), 1000.0, device="cuda").to(t)
        assert ((dq[0, 1, 0] - want).abs().float() <= U["bf16"] * 1000).all()


def test_qk_norm_rope_offsets_past_32_bits():
    """Rows further apart than 2^32 bytes."""
    torch = torch_mod()
    step = (1 << 31) + 64
    buf = torch.zeros(2 * step + 4096, dtype=torch.float16, device="cuda")
    big = buf.as_strided((3, 1, 2, 64), (step, 128, 64, 1))
    x = _draw(6, "big", (3, 1, 2, 64), "f16")[0]
    big.copy_(x)
    small = torch.ones(3, 1, 2, 64, dtype=torch.float16, device="cuda")
    ref = vg.qk_norm_rope(x, small)
    got = vg.qk_norm_rope(big, small, q_out=big)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    big.copy_(x)
    dref = vg.qk_norm_rope_backward(ref[0], small, x, small)
    dgot = vg.qk_norm_rope_backward(ref[0], small, big, small, dq=big)
    assert all(torch.equal(a, b) for a, b in zip(dgot, dref))


def test_qk_norm_rope_streams_and_captured_graphs():
    torch = torch_mod()
    case = (2, 300, 6, 2, 128, (16, 56, 56), "bf16", True, False, True, True)
    q, _, k, _, gq, _, gk, _, p, _, plan = _case(case)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    ref = (*vg.qk_norm_rope(q, k, gq, gk, p, plan), *vg.qk_norm_rope_backward(dq, dk, q, k, gq, gk, p, plan))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*vg.qk_norm_rope(q, k, gq, gk, p, plan, stream=side),
           *vg.qk_norm_rope_backward(dq, dk, q, k, gq, gk, p, plan, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # two graphs that share one workspace, replayed in turn
    ws = torch.empty(vg.qk_norm_rope_backward_workspace_bytes(2, 300, 6, 2, 128), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for gain in (1.0, 2.0):
        g = torch.cuda.CUDAGraph()
        a = dq * gain
        with torch.cuda.graph(g):
            outs.append(vg.qk_norm_rope_backward(a, dk, q, k, gq, gk, p, plan, workspace=ws))
        graphs.append((g, a))
    for _ in range(3):
        for g, _a in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], ref[2:]))
    assert torch.equal(outs[1][0], vg.qk_norm_rope_backward(dq * 2, dk, q, k, gq, gk, p, plan)[0])
    vg.sync_status()
