"""Oracle of the operators on latent tokens (float64): layer norm, rotary
positions, multi-head attention, and their gradients — test infrastructure only.

Written from the formulas alone, head by head and without any blocking. The
attention functions also return, on request, the sums of absolute values that
bound what roundings can do to each output (``bounds``)."""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def layernorm(x, gamma=None, beta=None, eps: float = 1e-6):
    """(x - mean) / sqrt(var + eps) * gamma + beta over the last axis, var biased."""
    x = _f64(x)
    d = x - x.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    if gamma is not None:
        y = y * _f64(gamma)
    return y if beta is None else y + _f64(beta)


def layernorm_backward(dy, x, gamma=None, eps: float = 1e-6):
    """(dx, dgamma, dbeta) of sum(dy * layernorm(x))."""
    x, dy = _f64(x), _f64(dy)
    d = x - x.mean(-1, keepdims=True)
    s = np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n = d / s
    g = dy if gamma is None else dy * _f64(gamma)
    dx = (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True)) / s
    return dx, (dy * n).sum(0), dy.sum(0)


def rope(x, positions, axes, theta: float = 10000.0, interleaved: bool = True, inverse: bool = False):
    """x [b][s][h][d]; positions [s][axes] or [b][s][axes]. Pairs of axis 0 first."""
    x, pos = _f64(x), _f64(positions)
    pos = np.broadcast_to(pos, x.shape[:2] + pos.shape[-1:])
    y = x.copy()
    rot = sum(axes)
    p = 0
    for a, n in enumerate(axes):
        for i in range(n // 2):
            ang = pos[..., a] * float(theta) ** (-2.0 * i / n)
            c, s = np.cos(ang)[..., None], np.sin(ang)[..., None]
            s = -s if inverse else s
            ia, ib = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
            y[..., ia] = x[..., ia] * c - x[..., ib] * s
            y[..., ib] = x[..., ia] * s + x[..., ib] * c
            p += 1
    return y


def seen(ql: int, kl: int, block: int):
    """[ql][kl] truth values: query i stands at i + kl - ql and sees its own block and the earlier ones."""
    if block == 0:
        return np.ones((ql, kl), bool)
    at = np.arange(ql) + kl - ql
    last = np.floor_divide(at, block)
    return (np.arange(kl) // block)[None] <= last[:, None]


def _entries(q, k, q_len, k_len):
    for e in range(q.shape[0]):
        ql = q.shape[1] if q_len is None else int(q_len[e])
        kl = k.shape[1] if k_len is None else int(k_len[e])
        yield e, ql, kl


def _softmax(q, k, scale, mask):
    s = scale * (q @ k.T)
    s = np.where(mask, s, -np.inf)
    top = s.max(1, initial=-np.inf)
    top = np.where(np.isinf(top), 0.0, top)
    p = np.exp(s - top[:, None])
    tot = p.sum(1)
    with np.errstate(divide="ignore"):
        lse = top + np.log(tot)
    return p / np.where(tot == 0, 1.0, tot)[:, None], lse


def attention(q, k, v, scale=None, q_len=None, k_len=None, block: int = 0, bounds: bool = False):
    """(o, lse) of q [b][sq][hq][d], k, v [b][sk][hkv][d]; rows behind q_len are 0 and -inf.
    bounds: also sum_j p |v| and the largest sum_c |q k| scale of each row's scores."""
    scale = 1.0 / np.sqrt(q.shape[-1]) if scale is None else scale
    b, sq, hq, d = q.shape
    g = hq // k.shape[2]
    o, lse = np.zeros(q.shape), np.full((b, hq, sq), -np.inf)
    pv, qk = np.zeros(q.shape), np.zeros((b, hq, sq))
    for e, ql, kl in _entries(q, k, q_len, k_len):
        m = seen(ql, kl, block)
        for h in range(hq):
            qq, kk, vv = _f64(q[e, :ql, h]), _f64(k[e, :kl, h // g]), _f64(v[e, :kl, h // g])
            p, lse[e, h, :ql] = _softmax(qq, kk, scale, m)
            o[e, :ql, h] = p @ vv
            if bounds:
                pv[e, :ql, h] = p @ np.abs(vv)
                qk[e, h, :ql] = scale * np.max(np.where(m, np.abs(qq) @ np.abs(kk).T, 0.0), 1, initial=0.0)
    return (o, lse, pv, qk) if bounds else (o, lse)


def attention_backward(do, q, k, v, scale=None, q_len=None, k_len=None, block: int = 0):
    """(dq, dk, dv) of sum(do * attention(q, k, v)); rows behind the lengths are 0."""
    scale = 1.0 / np.sqrt(q.shape[-1]) if scale is None else scale
    hq = q.shape[2]
    g = hq // k.shape[2]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for e, ql, kl in _entries(q, k, q_len, k_len):
        m = seen(ql, kl, block)
        for h in range(hq):
            qq, kk, vv = _f64(q[e, :ql, h]), _f64(k[e, :kl, h // g]), _f64(v[e, :kl, h // g])
            dd = _f64(do[e, :ql, h])
            p, _ = _softmax(qq, kk, scale, m)
            dp = dd @ vv.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            dq[e, :ql, h] = scale * ds @ kk
            dk[e, :kl, h // g] += scale * ds.T @ qq
            dv[e, :kl, h // g] += p.T @ dd
    return dq, dk, dv


def attention_backward_bounds(do, q, k, v, u, c, scale=None, q_len=None, k_len=None, block: int = 0, tiny=0.0,
                              exact_d: bool = False):
    """How far (dq, dk, dv) may be off, element by element, when probabilities and dS are rounded by u
    relative (and ``tiny`` absolute, times the largest |do| |v|), o carries 2 u of sum p |v|, and every
    sum in f32 carries c of its absolute values; without the outputs' own rounding. exact_d: rowsum(p dp)
    is formed from p and dp in f32 and not from the rounded o."""
    scale = 1.0 / np.sqrt(q.shape[-1]) if scale is None else scale
    hq = q.shape[2]
    g = hq // k.shape[2]
    eq, ek, ev = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    norm = lambda a: float(np.sqrt((np.nan_to_num(_f64(a)) ** 2).sum(-1)).max(initial=0.0))  # noqa: E731
    for e, ql, kl in _entries(q, k, q_len, k_len):
        m = seen(ql, kl, block)
        for h in range(hq):
            qq, kk, vv = _f64(q[e, :ql, h]), _f64(k[e, :kl, h // g]), _f64(v[e, :kl, h // g])
            dd = _f64(do[e, :ql, h])
            p, lse = _softmax(qq, kk, scale, m)
            dp = dd @ vv.T
            ad, av = np.abs(dd), np.abs(vv)
            D = (p * dp).sum(1, keepdims=True)
            x = np.abs(qq) @ np.abs(kk).T * scale
            ep = c * (1.0 + x + np.where(np.isinf(lse), 0.0, np.abs(lse))[:, None])  # of p, relative: exp of an f32 argument
            edp = c * (ad @ av.T)
            eD = (0.0 if exact_d else 2.0 * u) * (ad * (p @ av)).sum(1, keepdims=True) + c * (ad * (p @ av)).sum(1, keepdims=True)
            if exact_d:
                eD = eD + (p * (edp + ep * np.abs(dp))).sum(1, keepdims=True)
            ds = np.abs(p * (dp - D))
            eds = (u + 2 * c) * ds + p * (edp + eD + ep * np.abs(dp - D))
            eds = np.where(m, eds + tiny * norm(do) * norm(v), 0.0)
            ep = np.where(m, p * (ep + u) + tiny, 0.0)
            eq[e, :ql, h] = scale * (eds + c * ds) @ np.abs(kk)
            ek[e, :kl, h // g] += scale * (eds + c * ds).T @ np.abs(qq)
            ev[e, :kl, h // g] += (ep + c * p).T @ ad
    return eq, ek, ev


def qk_norm_rope(x, gamma=None, positions=None, axes=(), theta: float = 10000.0, interleaved: bool = True, eps: float = 1e-6):
    """One of the two tensors, x [b][s][h][d]: the norm of every head, its weight, the rotation."""
    x = _f64(x)
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if gamma is not None:
        z = z * _f64(gamma)
    return z if positions is None else rope(z, positions, axes, theta, interleaved)


def qk_norm_rope_backward(dy, x, gamma=None, positions=None, axes=(), theta: float = 10000.0, interleaved: bool = True,
                          eps: float = 1e-6):
    """(dx, dgamma) of sum(dy * qk_norm_rope(x))."""
    x, u = _f64(x), _f64(dy)
    if positions is not None:
        u = rope(u, positions, axes, theta, interleaved, inverse=True)
    size = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x / size
    v = u if gamma is None else u * _f64(gamma)
    return (v - n * (v * n).mean(-1, keepdims=True)) / size, (u * n).sum((0, 1, 2))


def activation(g, kind: str):
    """(act(g), its derivative)."""
    from scipy.special import erfc, expit
    g = _f64(g)
    if kind == "gelu":
        cdf = 0.5 * erfc(-g / np.sqrt(2.0))
        return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
    k, a = (1.0, 0.0) if kind == "silu" else (2.0 * np.sqrt(2.0 / np.pi), 0.044715)
    s = expit(k * (g + a * g ** 3))
    return g * s, s + g * s * expit(-k * (g + a * g ** 3)) * k * (1.0 + 3.0 * a * g * g)


def gated_ffn(x, w_gate, w_up, w_down, kind: str = "silu"):
    """(y, gate, up, hidden) of (act(x w_gate^T) * (x w_up^T)) w_down^T."""
    gate, up = _f64(x) @ _f64(w_gate).T, _f64(x) @ _f64(w_up).T
    hidden = activation(gate, kind)[0] * up
    return hidden @ _f64(w_down).T, gate, up, hidden


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, hidden, kind: str = "silu"):
    """(dx, dw_gate, dw_up, dw_down, dgate, dup) of sum(dy * y) at the given gate, up and hidden."""
    dy, x, up = _f64(dy), _f64(x), _f64(up)
    value, slope = activation(gate, kind)
    dh = dy @ _f64(w_down)
    dgate, dup = dh * up * slope, dh * value
    return dgate @ _f64(w_gate) + dup @ _f64(w_up), dgate.T @ x, dup.T @ x, dy.T @ _f64(hidden), dgate, dup
