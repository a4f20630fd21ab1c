"""GPU parity of the token operators against the float64 oracle: layer norm,
rotary positions, multi-head attention, and their gradients.

Tolerances are bounds, element by element, from the arithmetic alone:
- the rounding of the result to its type: half a step, U[type] of the value
  (2^-25 absolute in f16, whose steps stop shrinking below 2^-14);
- sums in f32: SUM = 2^-17 of the sum of absolute values, which covers up to
  128 roundings of 2^-24 along the longest chain of any sum here (128
  channels; partial sums of at most 64 rows or keys per chain, joined), twice
  over (2^-17 = 128 * 2^-24), and the 2-ulp exp, sqrt and divisions;
- attention's probabilities and dS in 16 bits: U of each, relative."""
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


def _t(name):
    torch = torch_mod()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _draw(seed, name, shape, t, std=1.0, mean=0.0):
    """A CUDA tensor of the type and its exact values in f64."""
    torch = torch_mod()
    a = rng_for(seed, "tok." + name).standard_normal(shape) * std + mean
    x = torch.from_numpy(np.ascontiguousarray(a)).to(_t(t)).cuda()
    return x, x.double().cpu().numpy()


def _np(x):
    return x.double().cpu().numpy()


def _within(got, ref, tol):
    got = _np(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == ref.shape
    assert not np.isnan(got).any()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


# ───────────────────────────── layer norm ─────────────────────────────

LN_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 33), (129, 144), (64, 256), (77, 257), (33, 576), (19, 1152), (18, 1280),
             (9, 1281), (7, 1288), (10, 2304), (6, 4096), (5, 5001), (4, 8192), (3, 16383), (3, 16384), (2500, 64),
             (5001, 144), (4900, 1152), (5000, 1280), (2600, 1288), (2500, 2560), (1300, 2568), (1400, 5120), (1300, 5128),
             (20003, 40), (20001, 200), (7300, 640), (4000, 648),
             (20011, 9), (20003, 35), (10001, 214), (5003, 1155), (3001, 2301), (1301, 5119)]


def _ln_terms(x, eps):
    """(n, rstd, how far n may be off)."""
    mean = x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    n = (x - mean) * rstd
    return n, rstd, rstd * SUM * (np.abs(x).mean(1, keepdims=True) + 2.0 ** -6 * np.abs(x)) + 2 * SUM * np.abs(n)


@pytest.mark.parametrize("m,c", LN_SHAPES)
@pytest.mark.parametrize("xt,yt,affine", [("f32", "f16", True), ("bf16", "bf16", True), ("f16", "f32", False),
                                          ("f32", "f32", True)])
def test_layernorm(m, c, xt, yt, affine):
    torch = torch_mod()
    x, x64 = _draw(1, f"ln.{m}.{c}", (m, c), xt, 2.0, 0.5)
    g, g64 = _draw(1, f"ln.g.{c}", (c,), "f32", 0.2, 1.0)
    b, b64 = _draw(1, f"ln.b.{c}", (c,), "f32", 0.2)
    out = torch.full((m, c), float("nan"), dtype=_t(yt), device="cuda")
    got = vg.layernorm(x, g if affine else None, b if affine else None, eps=1e-5, out=out)
    assert got is out
    ref = ot.layernorm(x64, g64 if affine else None, b64 if affine else None, 1e-5)
    n, _, en = _ln_terms(x64, 1e-5)
    ga = np.abs(g64) if affine else 1.0
    tol = U[yt] * np.abs(ref) * 1.001 + FLOOR[yt] + 1.01 * ga * en + (4 * U["f32"] * (np.abs(n) * ga + np.abs(ref)))
    _within(out, ref, tol)


def test_layernorm_in_place_constant_rows_and_one_operand():
    torch = torch_mod()
    x, x64 = _draw(2, "ln.inpl", (9, 72), "f16")
    ref = vg.layernorm(x)
    y = x.clone()
    assert vg.layernorm(y, out=y) is y and torch.equal(y, ref)
    z = vg.layernorm(torch.full((3, 40), 2.5, device="cuda"), beta=torch.arange(40.0, device="cuda"))
    assert torch.equal(z, torch.arange(40.0, device="cuda").expand(3, 40))
    g = torch.full((72,), 2.0, device="cuda")
    assert torch.equal(vg.layernorm(x, gamma=g, out_dtype=torch.float32), 2.0 * vg.layernorm(x, out_dtype=torch.float32))


def test_layernorm_odd_rows_off_the_boundaries():
    """Rows of an odd length from the second row of a tensor on: element by element, both directions."""
    torch = torch_mod()
    for m in (7, 20000):
        x, _ = _draw(2, f"ln.off.{m}", (m + 1, 33), "f16")
        dy, _ = _draw(2, f"ln.off.dy.{m}", (m + 1, 33), "f16")
        # (aligned and unaligned rows may take different forms: sums in another order, one more step of f16 at most)
        near = lambda a, b: (a.float() - b.float()).abs().max() <= 2.0 ** -9 * b.float().abs().max()  # noqa: E731
        assert near(vg.layernorm(x[1:]), vg.layernorm(x[1:].clone()))
        got, ref = vg.layernorm_backward(dy[1:], x[1:]), vg.layernorm_backward(dy[1:].clone(), x[1:].clone())
        assert near(got[0], ref[0])
        for a, b in zip(got[1:], ref[1:]):
            assert (a - b).abs().max() <= SUM * dy.float().abs().sum(0).max() * x.float().abs().max()


def test_layernorm_spikes_and_offsets():
    """A row far from zero and one with a single spike: the statistics are taken around the mean."""
    torch = torch_mod()
    r = rng_for(3, "tok.ln.spike").standard_normal((2, 512)).astype(np.float32)
    r[0] += 1000.0
    r[1, 0] = 5000.0
    x64 = r.astype(np.float64)
    n, _, en = _ln_terms(x64, 1e-6)
    _within(vg.layernorm(torch.from_numpy(r).cuda()), ot.layernorm(x64), 1.01 * en + 8 * U["f32"] * np.abs(n))


@pytest.mark.parametrize("m,c", LN_SHAPES)
@pytest.mark.parametrize("xt,dt,affine", [("f32", "f16", True), ("bf16", "bf16", True), ("f16", "f32", False),
                                          ("f32", "f32", True)])
def test_layernorm_backward(m, c, xt, dt, affine):
    torch = torch_mod()
    x, x64 = _draw(4, f"lnb.{m}.{c}", (m, c), xt, 2.0, 0.5)
    dy, dy64 = _draw(4, f"lnb.dy.{m}.{c}", (m, c), dt)
    g, g64 = _draw(4, f"lnb.g.{c}", (c,), "f32", 0.2, 1.0)
    eps = 1e-3
    nan = lambda *s, t: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    dx, dg, db = vg.layernorm_backward(dy, x, g if affine else None, eps=eps, dx=nan(m, c, t=_t(xt)),
                                       dgamma=nan(c, t=torch.float32), dbeta=nan(c, t=torch.float32))
    rx, rg, rb = ot.layernorm_backward(dy64, x64, g64 if affine else None, eps)
    n, rstd, en = _ln_terms(x64, eps)
    gr = np.abs(dy64 * (g64 if affine else 1.0))
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    m2 = np.abs(mean(dy64 * (g64 if affine else 1.0) * n))
    tol = U[xt] * np.abs(rx) * 1.001 + FLOOR[xt] + 2 * SUM * np.abs(rx) + 1.01 * rstd * (
        SUM * (2.0 ** -5 * gr + mean(gr) + 2 * np.abs(n) * mean(gr * np.abs(n))) + en * m2 + np.abs(n) * mean(gr * en))
    _within(dx, rx, tol)
    _within(dg, rg, (np.abs(dy64) * (1.01 * en + SUM * np.abs(n))).sum(0))
    _within(db, rb, SUM * np.abs(dy64).sum(0))
    again = vg.layernorm_backward(dy, x, g if affine else None, eps=eps)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dg) and torch.equal(again[2], db)
    only = vg.layernorm_backward(dy, x, g if affine else None, eps=eps, weight_grads=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None


def test_layernorm_backward_in_place():
    torch = torch_mod()
    x, _ = _draw(5, "lnb.inpl", (50, 1000), "f16")
    dy, _ = _draw(5, "lnb.inpl.dy", (50, 1000), "f16")
    ref = vg.layernorm_backward(dy, x)
    y = dy.clone()
    got = vg.layernorm_backward(y, x, dx=y)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    y = x.clone()
    got = vg.layernorm_backward(dy, y, dx=y)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_layernorm_backward_against_differences():
    """A gradient against central differences of the forward call itself: f32, a step of 2^-7 along random
    directions; the differences' own error is h^2 of the third derivative (under 1e-3 of the value here,
    |x| ~ 1, rstd ~ 1) and the rounding 2^-24 * 64 * sum / 2^-7 < 1e-3."""
    torch = torch_mod()
    x, _ = _draw(6, "lnb.diff", (4, 64), "f32")
    dy, dy64 = _draw(6, "lnb.diff.dy", (4, 64), "f32")
    g, _ = _draw(6, "lnb.diff.g", (64,), "f32", 0.2, 1.0)
    dx, dg, db = vg.layernorm_backward(dy, x, g)
    f = lambda xx, gg, bb: float((dy64 * _np(vg.layernorm(xx, gg, bb))).sum())  # noqa: E731
    h = 2.0 ** -7
    b = torch.zeros(64, device="cuda")
    for i in range(4):
        d, d64 = _draw(6, f"lnb.diff.d{i}", (4, 64), "f32", 0.2)
        num = (f(x + h * d, g, b) - f(x - h * d, g, b)) / (2 * h)
        assert abs(num - (d64 * _np(dx)).sum()) < 2e-2
        num = (f(x, g + h * d[0], b) - f(x, g - h * d[0], b)) / (2 * h)
        assert abs(num - (d64[0] * _np(dg)).sum()) < 2e-2
        num = (f(x, g, b + h * d[0]) - f(x, g, b - h * d[0])) / (2 * h)
        assert abs(num - (d64[0] * _np(db)).sum()) < 2e-2


# ───────────────────────────── rotary positions ─────────────────────────────

# b, s, h, d, axes, type, interleaved, int positions, per batch
ROPE = [(1, 1, 1, 2, (2,), "f32", True, True, False), (2, 5, 3, 10, (2, 6), "f16", False, False, True),
        (1, 256, 8, 64, (32, 32), "bf16", True, True, False), (2, 33, 6, 128, (16, 56, 56), "f16", True, False, True),
        (2, 33, 6, 128, (16, 56, 56), "bf16", False, True, False), (1, 700, 5, 96, (0, 32, 32), "f16", False, True, True),
        (3, 19, 2, 256, (64, 64, 64, 64), "f32", True, False, True), (1, 50, 4, 72, (8, 24, 24), "f32", False, True, False),
        (1, 50, 4, 66, (2, 32, 32), "f16", True, True, False), (2, 1000, 40, 40, (8, 16, 16), "bf16", True, False, True),
        (1, 9, 2, 256, (2,), "f16", True, True, False), (1, 700, 3, 255, (2,), "bf16", False, False, False), (2, 5, 2, 253, (100, 2, 0, 8), "f32", False, True, True)]


@pytest.mark.parametrize("case", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(case, inverse):
    torch = torch_mod()
    b, s, h, d, axes, t, inter, ints, per = case
    x, x64 = _draw(7, f"rope.{case}", (b, s, h, d), t)
    pos = rng_for(7, f"tok.rope.pos.{case}").integers(0, 1500, ((b, s) if per else (s,)) + (len(axes),))
    pos = pos if ints else pos + 0.25
    p = torch.from_numpy(np.asarray(pos, np.int32 if ints else np.float32)).cuda()
    plan = vg.RopePlan(axes, theta=10000.0, interleaved=inter)
    out = torch.full((b, s, h, d), float("nan"), dtype=_t(t), device="cuda")
    vg.rope(x, p, plan, inverse=inverse, out=out)
    ref = ot.rope(x64, pos, axes, 10000.0, inter, inverse)
    # the angle: a few 2^-24 turns; the turn: three roundings of terms up to |a| + |b| of the pair
    rot = sum(axes)
    pair = np.abs(ref).copy()
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    pair[..., ia] = pair[..., ib] = np.abs(x64[..., ia]) + np.abs(x64[..., ib])
    _within(out, ref, U[t] * np.abs(ref) * 1.001 + FLOOR[t] + 2.0 ** -20 * pair)
    assert torch.equal(out[..., rot:], x[..., rot:])
    y = x.clone()
    assert vg.rope(y, p, plan, inverse=inverse, out=y) is y and torch.equal(y, out)


def test_rope_far_positions_keep_their_angle():
    """Positions up to 2^24: the angle is off by a few 2^-24 turns (hi + lo carry 48 bits; pos * lo and
    the sum round once each: under 3 * 2^-24 turns, 2 pi of that in radians) and the turn as before."""
    torch = torch_mod()
    pos = np.array([[0], [1], [12345], [99991], [1 << 20], [(1 << 24) - 1], [-777]], np.float32)
    x, x64 = _draw(8, "rope.far", (1, 7, 2, 64), "f32")
    got = vg.rope(x, torch.from_numpy(pos).cuda(), vg.RopePlan((64,)))
    _within(got, ot.rope(x64, pos, (64,)), (2.0 ** -20 + 2.0 ** -19) * 2 * np.abs(x64).max() * np.ones(x64.shape))


def test_rope_views_of_a_joint_projection():
    """Queries and keys beside one another in one projection turn in one call; the values stay."""
    torch = torch_mod()
    qkv, q64 = _draw(9, "rope.view", (2, 40, 12, 64), "f16")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2).contiguous()
    plan = vg.RopePlan((32, 32))
    keep = qkv.clone()
    ref = vg.rope(keep[:, :, :8].contiguous(), pos, plan)
    vg.rope(qkv[:, :, :8], pos, plan, out=qkv[:, :, :8])
    assert torch.equal(qkv[:, :, :8], ref) and torch.equal(qkv[:, :, 8:], keep[:, :, 8:])
    # an odd channel offset: the element-by-element form
    wide = torch.zeros((2, 40, 8, 65), dtype=torch.float16, device="cuda")
    view = wide[..., 1:]
    vg.rope(keep[:, :, :8], pos, plan, out=view)
    assert torch.equal(view, ref) and not wide[..., 0].any()


# ───────────────────────────── attention ─────────────────────────────

# b, sq, sk, hq, hkv, d, type, block, q_len, k_len
ATT = [(1, 1, 1, 1, 1, 8, "f16", 0, None, None), (1, 1, 130, 2, 1, 64, "bf16", 0, None, None),
       (2, 127, 129, 2, 2, 40, "f16", 0, None, None), (1, 128, 128, 4, 4, 128, "bf16", 0, None, None),
       (1, 257, 300, 3, 1, 96, "f16", 0, None, None), (2, 256, 256, 8, 8, 64, "f16", 0, None, None),
       (1, 200, 200, 4, 2, 128, "f16", 1, None, None), (1, 300, 300, 6, 1, 72, "bf16", 64, None, None),
       (1, 5, 700, 16, 4, 128, "bf16", 1, None, None), (1, 700, 90, 2, 2, 64, "f16", 16, None, None),
       (4, 1, 2000, 16, 4, 128, "bf16", 0, None, [2000, 1, 0, 777]), (4, 1, 999, 8, 1, 64, "f16", 7, None, [5, 999, 128, 129]),
       (3, 150, 160, 4, 2, 80, "f16", 0, [150, 0, 1], [160, 33, 0]), (3, 310, 310, 4, 4, 128, "bf16", 100, [310, 7, 131], [310, 9, 256]),
       (2, 64, 64, 12, 4, 16, "bf16", 3, [60, 64], [64, 20]), (1, 1100, 1100, 2, 1, 120, "f16", 0, None, None),
       (1, 3, 5000, 32, 2, 128, "f16", 1, None, None), (2, 513, 640, 5, 5, 24, "bf16", 50, [400, 513], [640, 100]),
       # enough tiles for every SM: tiles in pairs, an odd one left over
       (4, 300, 310, 40, 40, 32, "f16", 0, [300, 0, 129, 1], [310, 128, 7, 300]),
       (2, 1200, 1200, 16, 8, 64, "bf16", 70, [1200, 1030], [1200, 1100]), (1, 1300, 1300, 16, 16, 128, "f16", 1, None, None),
       (1, 640, 1290, 40, 40, 128, "bf16", 0, None, [1290]), (3, 130, 258, 64, 64, 96, "f16", 33, [130, 128, 64], [258, 200, 129])]


def _att_inputs(case, seed=11):
    torch = torch_mod()
    b, sq, sk, hq, hkv, d, t, block, q_len, k_len = case
    q, q64 = _draw(seed, f"att.q.{case}", (b, sq, hq, d), t, 1.5)
    k, k64 = _draw(seed, f"att.k.{case}", (b, sk, hkv, d), t)
    v, v64 = _draw(seed, f"att.v.{case}", (b, sk, hkv, d), t)
    do, do64 = _draw(seed, f"att.do.{case}", (b, sq, hq, d), t)
    # what lies behind the lengths may be anything
    for x, n in ((q, q_len), (do, q_len), (k, k_len), (v, k_len)):
        if n is not None:
            for e, m in enumerate(n):
                x[e, m:] = float("nan")
                x[e, m::3] = float("inf")
    i32 = lambda n: None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return (q, k, v, do), (q64, k64, v64, do64), dict(q_len=i32(q_len), k_len=i32(k_len), block=block), \
        dict(q_len=q_len, k_len=k_len, block=block)


def _rows_behind(case):
    """[b][sq] truth values of the query rows behind q_len, and [b][sk] of the keys behind k_len."""
    b, sq, sk, q_len, k_len = case[0], case[1], case[2], case[8], case[9]
    ql = np.full(b, sq) if q_len is None else np.array(q_len)
    kl = np.full(b, sk) if k_len is None else np.array(k_len)
    return np.arange(sq)[None] >= ql[:, None], np.arange(sk)[None] >= kl[:, None]


@pytest.mark.parametrize("case", ATT)
def test_attention(case):
    torch = torch_mod()
    t = case[6]
    (q, k, v, _), (q64, k64, v64, _), kw, okw = _att_inputs(case)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((case[0], case[3], case[1]), 7.0, device="cuda")
    o, l = vg.attention(q, k, v, out=out, lse=lse, **kw)
    vg.sync_status()
    ro, rl, pv, qk = ot.attention(q64, k64, v64, bounds=True, **okw)
    behind, _ = _rows_behind(case)
    # rows behind the lengths are left as they were
    assert (_np(o)[behind] == 7.0).all() and (_np(l).transpose(0, 2, 1)[behind] == 7.0).all()
    gl, go = _np(l), _np(o)
    valid = ~behind
    gl, rl = gl.transpose(0, 2, 1)[valid], rl.transpose(0, 2, 1)[valid]
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty).all() and (go[valid][empty] == 0.0).all()
    es = SUM * (1.0 + qk.transpose(0, 2, 1)[valid] + np.where(empty, 0.0, np.abs(rl)))  # of a score, and so of p, relative
    _within(gl[~empty], rl[~empty], 2 * es[~empty])
    ro, pv = ro[valid], pv[valid]
    _within(go[valid], ro, U[t] * np.abs(ro) * 1.001 + FLOOR[t] + (U[t] + 2 * es[..., None] + SUM) * pv + 2.0 ** -24 * pv.max())
    o2, l2 = vg.attention(q, k, v, **kw)
    assert torch.equal(o2[torch.from_numpy(valid).cuda()], o[torch.from_numpy(valid).cuda()])
    assert not o2[torch.from_numpy(behind).cuda()].any()
    assert torch.isneginf(l2.transpose(1, 2)[torch.from_numpy(behind).cuda()]).all()


@pytest.mark.parametrize("case", ATT)
def test_attention_backward(case):
    torch = torch_mod()
    t = case[6]
    (q, k, v, do), (q64, k64, v64, do64), kw, okw = _att_inputs(case)
    o, lse = vg.attention(q, k, v, **kw)
    full = lambda x: torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")  # noqa: E731
    got = vg.attention_backward(do, q, k, v, o, lse, dq=full(q), dk=full(k), dv=full(v), **kw)
    vg.sync_status()
    ref = ot.attention_backward(do64, q64, k64, v64, **okw)
    # 2^-39: P and dS in f16 are held scaled so that a step below 2^-14 is that small against the largest
    tol = ot.attention_backward_bounds(do64, q64, k64, v64, U[t], SUM, tiny=2.0 ** -38 if t == "f16" else 2.0 ** -100, **okw)
    rows, keys = _rows_behind(case)
    for g, r, e, behind in zip(got, ref, tol, (rows, keys, keys)):
        gg = _np(g)
        assert (gg[behind] == 7.0).all()
        _within(gg[~behind], r[~behind], 1.01 * e[~behind] + U[t] * np.abs(r[~behind]) * 1.001 + FLOOR[t])
    again = vg.attention_backward(do, q, k, v, o, lse, **kw)
    for g, a, behind in zip(got, again, (rows, keys, keys)):
        m = torch.from_numpy(behind).cuda()
        assert torch.equal(a[~m], g[~m]) and not a[m].any()


@pytest.mark.parametrize("gain", [2.0 ** -12, 2.0 ** -6, 2.0 ** 6])
def test_attention_backward_f16_gradients_of_any_size(gain):
    """Small and large incoming gradients in f16: dS has a scale of its own. The bound's tiny term is
    relative to the largest |do| |v|, and dq, dk here are far above the smallest f16 steps (gain 2^-12:
    their own rounding floor 2^-25 is in the bound)."""
    case = (1, 300, 333, 2, 2, 64, "f16", 0, None, None)
    (q, k, v, do), (q64, k64, v64, _), kw, okw = _att_inputs(case)
    do = (do.float() * gain).half()
    do64 = _np(do)
    o, lse = vg.attention(q, k, v, **kw)
    got = vg.attention_backward(do, q, k, v, o, lse, **kw)
    vg.sync_status()
    ref = ot.attention_backward(do64, q64, k64, v64, **okw)
    tol = ot.attention_backward_bounds(do64, q64, k64, v64, U["f16"], SUM, tiny=2.0 ** -38, **okw)
    for g, r, e in zip(got, ref, tol):
        _within(g, r, 1.01 * e + U["f16"] * np.abs(r) * 1.001 + FLOOR["f16"])


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_attention_peaked_scores(t):
    """Scores up to hundreds: the running maximum moves far, late keys win."""
    torch = torch_mod()
    case = (1, 130, 1000, 2, 2, 64, t, 0, None, None)
    (q, k, v, do), (_, _, v64, do64), kw, okw = _att_inputs(case)
    grow = torch.linspace(0.1, 6.0, 1000, device="cuda")[None, :, None, None]
    q, k = (q.float() * 4).to(q.dtype), (k.float() * grow).to(k.dtype)
    q64, k64 = _np(q), _np(k)
    o, lse = vg.attention(q, k, v, **kw)
    ro, rl, pv, qk = ot.attention(q64, k64, v64, bounds=True, **okw)
    es = SUM * (1.0 + qk + np.abs(rl)).transpose(0, 2, 1)[..., None]
    _within(lse, rl, 2 * es[..., 0].transpose(0, 2, 1))
    _within(o, ro, U[t] * np.abs(ro) * 1.001 + FLOOR[t] + (U[t] + 2 * es + SUM) * pv + 2.0 ** -24 * pv.max())
    got = vg.attention_backward(do, q, k, v, o, lse, **kw)
    ref = ot.attention_backward(do64, q64, k64, v64, **okw)
    tol = ot.attention_backward_bounds(do64, q64, k64, v64, U[t], SUM, tiny=2.0 ** -38 if t == "f16" else 2.0 ** -100, **okw)
    for g, r, e in zip(got, ref, tol):
        _within(g, r, 1.01 * e + U[t] * np.abs(r) * 1.001 + FLOOR[t])


FEW = [
    # b, sq, sk, hq, hkv, d, type, block, q_len, k_len: at most 64 rows of a key head (the output: 16)
    (2, 1, 16, 4, 2, 64, "bf16", 0, None, None),
    (1, 5, 20, 3, 3, 64, "f16", 0, None, None),
    (1, 30, 30, 2, 2, 128, "bf16", 1, None, None),
    (1, 30, 200, 2, 1, 72, "f16", 0, None, None),
    (2, 16, 200, 2, 2, 96, "f16", 0, (7, 16), (200, 90)),
    (2, 64, 256, 2, 2, 64, "bf16", 16, (64, 41), None),
    (2, 1, 3001, 8, 2, 128, "f16", 0, None, (3001, 17)),
    (1, 3, 1500, 4, 4, 64, "bf16", 0, None, None),
    (1, 4, 700, 24, 2, 40, "bf16", 0, None, None),  # 12 heads to a key head: three parts of four
]


@pytest.mark.parametrize("case", FEW)
def test_attention_few_rows_in_two_parts(case):
    """Few rows lie twice in a tile, and P and dS are held in two 16-bit parts: what the second rounds off is at most U of the
    first's U, so that the results are off by their own rounding and U U of the sums only (gradients of
    scores where D is formed from f32, up to 256 keys; f16's second part, 2^-14 of the first's scale at
    the least, ends at 2^-25 2^-14, under the bound's tiny term)."""
    t = case[6]
    (q, k, v, do), (q64, k64, v64, do64), kw, okw = _att_inputs(case)
    o, lse = vg.attention(q, k, v, **kw)
    got = vg.attention_backward(do, q, k, v, o, lse, **kw)
    vg.sync_status()
    rows, keys = _rows_behind(case)
    ro, rl, pv, qk = ot.attention(q64, k64, v64, bounds=True, **okw)
    es = SUM * (1.0 + qk + np.where(np.isinf(rl), 0.0, np.abs(rl))).transpose(0, 2, 1)[..., None]
    tol = U[t] * np.abs(ro) * 1.001 + FLOOR[t] + (U[t] ** 2 + 2 * es + SUM) * pv + 2.0 ** -38 * pv.max()
    gp = np.gcd(case[3] // case[4], 64)
    if case[1] * gp <= 16:
        _within(_np(o)[~rows], ro[~rows], tol[~rows])
    ref = ot.attention_backward(do64, q64, k64, v64, **okw)
    tol = ot.attention_backward_bounds(do64, q64, k64, v64, U[t] ** 2, SUM, tiny=2.0 ** -38 if t == "f16" else 2.0 ** -100, **okw)
    for n, (g, r, e, behind) in enumerate(zip(got, ref, tol, (rows, keys, keys))):
        if n == 2 or case[2] <= 256:
            _within(_np(g)[~behind], r[~behind], 1.01 * e[~behind] + U[t] * np.abs(r[~behind]) * 1.001 + FLOOR[t])


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("case", [(2, 1, 1, 4, 2, 64, 1, None), (1, 300, 1, 3, 3, 128, 0, None), (2, 140, 50, 4, 1, 96, 0, (1, 1)),
                                  (1, 1, 1, 1, 1, 40, 0, None)])
def test_attention_single_key(case, t):
    """Softmax over one key is 1 whatever its score: o is the value, dq and dk are exactly 0."""
    torch = torch_mod()
    b, sq, sk, hq, hkv, d, block, k_len = case
    (q, k, v, do), (_, _, _, do64), kw, _ = _att_inputs((b, sq, sk, hq, hkv, d, t, block, None, k_len))
    o, lse = vg.attention(q, k, v, **kw)
    dq, dk, dv = vg.attention_backward(do, q, k, v, o, lse, **kw)
    vg.sync_status()
    assert torch.equal(o, v[:, :1].repeat_interleave(hq // hkv, 2).expand_as(o))
    assert not dq.any() and not dk.any()
    ref = do64.reshape(b, sq, hkv, hq // hkv, d)
    tol = (U[t] ** 2 + 2 * SUM) * np.abs(ref).sum((1, 3))
    _within(dv[:, 0], ref.sum((1, 3)), tol * 1.01 + U[t] * np.abs(ref.sum((1, 3))) * 1.001 + FLOOR[t])


def test_attention_strided_views_and_other_token_orders():
    """q, k, v as views of one projection, outputs and gradients into views, batch and token dims swapped
    in memory: the same bits as with dense tensors."""
    torch = torch_mod()
    b, s, h, d = 2, 190, 4, 64
    qkv, _ = _draw(12, "att.view", (s, b, 3 * h, d), "bf16")
    x = qkv.transpose(0, 1)  # [b][s][3h][d], token stride over the batch's
    q, k, v = x[:, :, :h], x[:, :, h:2 * h], x[:, :, 2 * h:]
    do, _ = _draw(12, "att.view.do", (b, h, s, d), "bf16")
    do = do.transpose(1, 2)  # heads before tokens in memory
    o, lse = vg.attention(q, k, v, block=10)
    dense = [a.contiguous() for a in (q, k, v)]
    ro, rl = vg.attention(*dense, block=10)
    assert torch.equal(o, ro) and torch.equal(lse, rl)
    wide = torch.full((b, s, 3 * h, d), 7.0, dtype=q.dtype, device="cuda")
    dq, dk, dv = wide[:, :, :h], wide[:, :, h:2 * h], wide[:, :, 2 * h:]
    vg.attention_backward(do, q, k, v, o, lse, block=10, dq=dq, dk=dk, dv=dv)
    ref = vg.attention_backward(do.contiguous(), *dense, ro, rl, block=10)
    for a, r in zip((dq, dk, dv), ref):
        assert torch.equal(a, r)


def test_attention_scale_and_lengths_out_of_range_are_clamped():
    torch = torch_mod()
    case = (2, 40, 50, 2, 2, 64, "f16", 0, None, None)
    (q, k, v, _), (q64, k64, v64, _), _, _ = _att_inputs(case)
    far = torch.tensor([1000, -5], dtype=torch.int32, device="cuda")
    o, lse = vg.attention(q, k, v, scale=0.01, k_len=far)
    ref, _ = vg.attention(q, k, v, scale=0.01)
    assert torch.equal(o[0], ref[0]) and not o[1].any() and torch.isneginf(lse[1]).all()
    ro, _, pv, qk = ot.attention(q64, k64, v64, scale=0.01, bounds=True)
    _within(ref, ro, U["f16"] * np.abs(ro) + FLOOR["f16"] + (U["f16"] + SUM * (4 + 2 * qk.max())) * pv * 1.01 + 2.0 ** -24 * pv.max())


def test_attention_new_tensors_beside_given_ones():
    """Rows behind the lengths: left in a tensor that the caller gave, 0 (lse -inf) in new ones, whichever are given."""
    torch = torch_mod()
    case = (3, 150, 160, 4, 2, 80, "f16", 0, [150, 0, 1], [160, 33, 0])
    (q, k, v, do), _, kw, _ = _att_inputs(case)
    rows, keys = (torch.from_numpy(m).cuda() for m in _rows_behind(case))
    o, lse = vg.attention(q, k, v, **kw)
    o1, l1 = vg.attention(q, k, v, out=torch.full_like(q, 7.0), **kw)
    assert torch.equal(l1, lse) and (o1[rows] == 7.0).all() and torch.equal(o1[~rows], o[~rows]) and not o[rows].any()
    o2, l2 = vg.attention(q, k, v, lse=torch.full_like(lse, 7.0), **kw)
    assert torch.equal(o2, o) and (l2.transpose(1, 2)[rows] == 7.0).all()
    dq, dk, dv = vg.attention_backward(do, q, k, v, o, lse, **kw)
    dq1, dk1, dv1 = vg.attention_backward(do, q, k, v, o, lse, dk=torch.full_like(k, 7.0), **kw)
    assert torch.equal(dq1, dq) and torch.equal(dv1, dv) and (dk1[keys] == 7.0).all() and torch.equal(dk1[~keys], dk[~keys])
    assert not dq[rows].any() and not dk[keys].any() and not dv[keys].any()


def test_attention_offsets_past_32_bits():
    """The second batch entry's keys lie over 2^31 elements behind the first's."""
    torch = torch_mod()
    sk, hkv, d = 300, 2, 64
    gap = (1 << 31) + 4096
    buf = torch.empty(gap + 2 * sk * hkv * d, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((2, sk, hkv, d), (gap, hkv * d, d, 1))
    v = buf.as_strided((2, sk, hkv, d), (gap, hkv * d, d, 1), sk * hkv * d)
    (q, k0, v0, do), _, _, _ = _att_inputs((2, 70, sk, 4, hkv, d, "bf16", 0, None, None))
    k.copy_(k0)
    v.copy_(v0)
    o, lse = vg.attention(q, k, v)
    ro, rl = vg.attention(q, k0, v0)
    assert torch.equal(o, ro) and torch.equal(lse, rl)
    for a, r in zip(vg.attention_backward(do, q, k, v, o, lse), vg.attention_backward(do, q, k0, v0, ro, rl)):
        assert torch.equal(a, r)


def test_attention_streams_and_captured_graphs():
    """Two calls at once on streams of their own, and one captured with its gradient and replayed on new
    inputs: the same bits as eager calls."""
    torch = torch_mod()
    case = (2, 300, 400, 8, 2, 128, "bf16", 0, None, None)
    (q, k, v, do), _, _, _ = _att_inputs(case)
    o, lse = vg.attention(q, k, v)
    ref = vg.attention_backward(do, q, k, v, o, lse)
    q1 = q[:, :1].contiguous()
    o1, _ = vg.attention(q1, k, v)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a = [vg.attention(q, k, v, stream=s1) for _ in range(4)]
    c = [vg.attention(q1, k, v, stream=s2) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], o) and torch.equal(x[1], lse) for x in a) and all(torch.equal(x[0], o1) for x in c)
    static = [x.clone() for x in (q, k, v, do)]
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        go, gl = vg.attention(*static[:3])
        grads = vg.attention_backward(static[3], *static[:3], go, gl)
    for x, y in zip(static, (q, k, v, do)):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(go, o) and all(torch.equal(x, y) for x, y in zip(grads, ref))
    static[0].copy_(q.flip(1))
    g.replay()
    o2, l2 = vg.attention(q.flip(1).contiguous(), k, v)
    assert torch.equal(go, o2) and torch.equal(gl, l2)


def test_operators_launched_ahead():
    """With every kernel launched while the one before it still runs (VAE_PDL=1, read once per process): the same
    results, as each waits for the grid before it."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", os.path.abspath(__file__),
                        "-k", "strided_views or together or test_token_block or peaked or joint or in_place"],
                       cwd=root, env=dict(os.environ, VAE_PDL="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


# ───────────────────────────── together ─────────────────────────────

def test_token_block_forward_and_backward():
    """norm -> q, k, v projections -> rotary positions -> attention over frames -> output projection with the
    residual, and the gradient back to the input, through the library's own calls; against float64.
    At most a dozen roundings of half an f16 step (2^-11) lie between input and output in either direction,
    and roundings of q and k move scores of a few units by 2^-11 each, p by 2^-8 at most: 2^-7 of the norm."""
    torch = torch_mod()
    b, f, s, h, d = 2, 3, 50, 4, 32
    c, n, block = h * d, f * s, s
    m = b * n
    x, x64 = _draw(20, "blk.x", (m, c), "f32")
    gam, g64 = _draw(20, "blk.g", (c,), "f32", 0.2, 1.0)
    bet, b64 = _draw(20, "blk.b", (c,), "f32", 0.2)
    w, w64 = {}, {}
    for i in "qkvo":
        w[i], w64[i] = _draw(20, "blk.w" + i, (c, c), "f16", 1.0 / np.sqrt(c))
    dy, dy64 = _draw(20, "blk.dy", (m, c), "f16")
    grid = torch.stack(torch.meshgrid(torch.arange(f), torch.arange(5), torch.arange(10), indexing="ij"), -1).reshape(n, 3)
    pos = grid.to(torch.int32).cuda()
    axes = (8, 12, 12)
    plan = vg.RopePlan(axes)
    heads = lambda a: a.view(b, n, h, d)  # noqa: E731
    # forward
    y = vg.layernorm(x, gam, bet, out_dtype=torch.float16)
    q, k, v = (heads(vg.conv1x1(y, w[i], out_f16=True)) for i in "qkv")
    q, k = vg.rope(q, pos, plan), vg.rope(k, pos, plan)
    o, lse = vg.attention(q, k, v, block=block)
    out = vg.conv1x1(o.view(m, c), w["o"], residual=x)
    # backward
    wt = {i: w[i].t().contiguous() for i in w}
    do = heads(vg.conv1x1(dy, wt["o"], out_f16=True))
    dq, dk, dv = vg.attention_backward(do, q, k, v, o, lse, block=block)
    dq, dk = vg.rope(dq, pos, plan, inverse=True), vg.rope(dk, pos, plan, inverse=True)
    dn = None
    for i, t in (("q", dq), ("k", dk), ("v", dv)):
        dn = vg.conv1x1(t.view(m, c), wt[i], residual=dn)
    dx, dgam, dbet = vg.layernorm_backward(dn, x, gam)
    vg.sync_status()
    # float64
    yr = ot.layernorm(x64, g64, b64)
    qr, kr, vr = ((yr @ w64[i].T).reshape(b, n, h, d) for i in "qkv")
    p = grid.numpy()
    qr, kr = ot.rope(qr, p, axes), ot.rope(kr, p, axes)
    orr, _ = ot.attention(qr, kr, vr, block=block)
    outr = orr.reshape(m, c) @ w64["o"].T + x64
    dor = (dy64 @ w64["o"]).reshape(b, n, h, d)
    dqr, dkr, dvr = ot.attention_backward(dor, qr, kr, vr, block=block)
    dqr, dkr = ot.rope(dqr, p, axes, inverse=True), ot.rope(dkr, p, axes, inverse=True)
    dnr = sum(a.reshape(m, c) @ w64[i] for i, a in (("q", dqr), ("k", dkr), ("v", dvr)))
    dxr, dgr, dbr = ot.layernorm_backward(dnr, x64, g64)
    off = lambda a, r: np.linalg.norm(_np(a) - r) / np.linalg.norm(r)  # noqa: E731
    assert off(out, outr) <= 2.0 ** -7
    assert off(dx, dxr) <= 2.0 ** -7 and off(dgam, dgr) <= 2.0 ** -7 and off(dbet, dbr) <= 2.0 ** -7
