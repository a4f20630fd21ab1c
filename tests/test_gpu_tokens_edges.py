"""GPU parity of the token operators where the values or the shapes are unusual.
Oracle, tolerances and inputs as in test_gpu_tokens.py."""
import numpy as np
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
import test_gpu_tokens as base
from gpu_common import torch_mod
from oracle import tokens as ot
from test_gpu_tokens import FLOOR, SUM, U, _att_inputs, _draw, _ln_terms, _np, _within

pytestmark = pytest.mark.gpu

# ───────────────────────────── NaN that counts ─────────────────────────────

# the forms of the forward: b, sq, sk, hq, hkv, d, type, block, q_len, k_len
NAN_FORMS = [
    (1, 4, 100, 4, 4, 64, "f16", 0, None, None),                  # at most 32 rows, one key tile
    (2, 1, 300, 8, 2, 128, "bf16", 0, None, None),                # at most 32 rows, both streams
    (2, 1, 3000, 8, 2, 128, "bf16", 0, None, [2945, 700]),        # at most 32 rows, keys over CTAs
    (1, 24, 2000, 1, 1, 96, "f16", 0, None, None),                # the same, rows once a quadrant
    (1, 100, 100, 2, 2, 64, "f16", 0, None, None),                # one row tile, one stream
    (1, 100, 300, 2, 2, 128, "bf16", 1, None, None),              # one row tile, both streams
    (1, 100, 3000, 3, 1, 64, "f16", 0, None, [2945]),             # one row tile, keys over CTAs
    (4, 300, 310, 40, 40, 32, "f16", 0, [300, 0, 129, 1], [310, 128, 7, 300]),  # row tiles in pairs
]


def _nan_call(case, q, k, v, kw, okw):
    """(o, lse, the oracle's o and lse) of a call, and the check that NaN stands where the oracle's does."""
    o, lse = vg.attention(q, k, v, **kw)
    vg.sync_status()
    with np.errstate(invalid="ignore"):
        ro, rl = ot.attention(_np(q), _np(k), _np(v), **okw)
    assert (np.isnan(_np(o)) == np.isnan(ro)).all()
    assert (np.isnan(_np(lse)) == np.isnan(rl)).all() and (np.isneginf(_np(lse)) == np.isneginf(rl)).all()
    return o, lse, ro, rl


@pytest.mark.parametrize("case", NAN_FORMS)
@pytest.mark.parametrize("where", ["query", "key", "last key"])
def test_attention_nan_in_rows_and_keys_that_count(case, where):
    """NaN in a valid query row is NaN in its output and log-sum-exp, NaN in a key is NaN for the rows that see it,
    and the rows that meet neither keep their bits."""
    torch = torch_mod()
    b, sq, sk, hq, hkv, _, _, _, q_len, k_len = case
    (q, k, v, _), _, kw, okw = _att_inputs(case)
    clean, clean_lse = vg.attention(q, k, v, **kw)
    kl = sk if k_len is None else k_len[0]
    q, k = q.clone(), k.clone()
    if where == "query":
        i = (sq if q_len is None else q_len[0]) - 1
        q[0, i, hq - 1, 3] = float("nan")
        q[0, i // 2, 0] = float("nan")
    else:
        k[0, kl - 1 if where == "last key" else kl // 3, hkv - 1, 5] = float("nan")
    o, lse, ro, rl = _nan_call(case, q, k, v, kw, okw)
    met = torch.from_numpy(np.isnan(rl)).cuda()
    assert met.any() and torch.equal(lse[~met], clean_lse[~met])
    met = met.transpose(1, 2)
    assert torch.equal(o[~met], clean[~met])


def test_attention_nan_piece_of_one_key():
    """A split whose only key holds NaN: its part joins as NaN."""
    case = (1, 1, 1300, 4, 1, 64, "f16", 0, None, None)
    (q, k, v, _), _, _, _ = _att_inputs(case)
    torch = torch_mod()
    for kl in (1, 129, 257, 1025, 1281):
        n = torch.tensor([kl], dtype=torch.int32, device="cuda")
        kk = k.clone()
        kk[0, kl - 1, 0, 0] = float("nan")
        o, lse = vg.attention(q, kk, v, k_len=n)
        assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("case", [(1, 4, 100, 4, 4, 64, "f16", 0, None, None), (1, 140, 600, 4, 2, 128, "bf16", 0, None, None)])
def test_attention_backward_nan_row(case):
    """The gradient of a query row with NaN is NaN in its dq and, as every key meets the row, in its head's dk and dv;
    the other rows' dq keep their bits."""
    torch = torch_mod()
    hq, hkv = case[3], case[4]
    (q, k, v, do), _, kw, _ = _att_inputs(case)
    o, lse = vg.attention(q, k, v, **kw)
    ref = vg.attention_backward(do, q, k, v, o, lse, **kw)
    q = q.clone()
    q[0, 2, hq - 1, 7] = float("nan")
    o, lse = vg.attention(q, k, v, **kw)
    dq, dk, dv = vg.attention_backward(do, q, k, v, o, lse, **kw)
    vg.sync_status()
    assert torch.isnan(dq[0, 2, hq - 1]).all()
    dq[0, 2, hq - 1] = ref[0][0, 2, hq - 1]
    assert torch.equal(dq, ref[0])
    for a, r in ((dk, ref[1]), (dv, ref[2])):
        assert torch.isnan(a[:, :, hkv - 1]).all() and torch.equal(a[:, :, :hkv - 1], r[:, :, :hkv - 1])


# ───────────────────────────── layer norm ─────────────────────────────

@pytest.mark.parametrize("m,c", [(1, 64), (64, 256), (15001, 144), (15002, 144), (4901, 1152), (20003, 35), (20001, 200), (1401, 5120)])
def test_layernorm_backward_without_eps(m, c):
    """eps 0, which is allowed, and row counts that end inside a chunk: the rows that are not there count nothing."""
    x, x64 = _draw(29, f"ln.eps0.{m}.{c}", (m, c), "f32", 1.0, 0.25)
    dy, dy64 = _draw(29, f"ln.eps0.dy.{m}.{c}", (m, c), "f16")
    n, rstd, en = _ln_terms(x64, 0.0)
    dx, dg, db = vg.layernorm_backward(dy, x, eps=0.0)
    rx, rg, rb = ot.layernorm_backward(dy64, x64, None, 0.0)
    gr = np.abs(dy64)
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    m2 = np.abs(mean(dy64 * n))
    _within(dx, rx, U["f32"] * np.abs(rx) * 1.001 + 2 * SUM * np.abs(rx) + 1.01 * rstd * (
        SUM * (2.0 ** -5 * gr + mean(gr) + 2 * np.abs(n) * mean(gr * np.abs(n))) + en * m2 + np.abs(n) * mean(gr * en)))
    _within(dg, rg, (gr * (1.01 * en + SUM * np.abs(n))).sum(0))
    _within(db, rb, SUM * gr.sum(0))


@pytest.mark.parametrize("m,c", [(64, 256), (5001, 144), (4900, 1152), (20003, 35), (1400, 5120)])
@pytest.mark.parametrize("log2", [-52, 52])
def test_layernorm_of_values_far_from_one(m, c, log2):
    """Rows 2^52 and 2^-52 large: the statistics' squares stay within f32, and so does everything formed
    from them. The bounds are those of values near one, which scale with the rows."""
    x, x64 = _draw(30, f"ln.far.{m}.{c}.{log2}", (m, c), "f32", 2.0 ** log2, 2.0 ** (log2 - 2))
    dy, dy64 = _draw(30, f"ln.far.dy.{m}.{c}", (m, c), "f32")
    g, g64 = _draw(30, f"ln.far.g.{c}", (c,), "f32", 0.2, 1.0)
    n, rstd, en = _ln_terms(x64, 0.0)
    ref = ot.layernorm(x64, g64, None, 0.0)
    _within(vg.layernorm(x, g, eps=0.0), ref, 1.01 * np.abs(g64) * en + 8 * U["f32"] * np.abs(ref))
    dx, dg, db = vg.layernorm_backward(dy, x, g, eps=0.0)
    rx, rg, rb = ot.layernorm_backward(dy64, x64, g64, 0.0)
    gr = np.abs(dy64 * g64)
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    m2 = np.abs(mean(dy64 * g64 * n))
    tol = U["f32"] * np.abs(rx) * 1.001 + 2 * SUM * np.abs(rx) + 1.01 * rstd * (
        SUM * (2.0 ** -5 * gr + mean(gr) + 2 * np.abs(n) * mean(gr * np.abs(n))) + en * m2 + np.abs(n) * mean(gr * en))
    _within(dx, rx, tol)
    _within(dg, rg, (np.abs(dy64) * (1.01 * en + SUM * np.abs(n))).sum(0))
    _within(db, rb, SUM * np.abs(dy64).sum(0))


# ───────────────────────────── gradients far apart ─────────────────────────────

@pytest.mark.parametrize("case", [(2, 300, 333, 2, 2, 64, "f16", 0, None, None), (2, 20, 200, 4, 2, 64, "f16", 0, None, None)])
@pytest.mark.parametrize("small", ["entry", "head"])
def test_attention_backward_f16_sizes_apart(case, small):
    """One entry's (or key head's) do and v 2^24 under the other's, in f16: its gradients keep their digits, as if it
    were alone in the call. Bounds: those of a call of its own (the tiny term is relative to its own
    largest |do| |v|); keys times eight put its dq over f16's smallest steps."""
    (q, k, v, do), _, _, _ = _att_inputs(case)
    k = (k.float() * 8).half()
    q = (q.float() / 8).half()
    g = case[3] // case[4]
    big = (slice(0, 1), slice(None)) if small == "entry" else (slice(None), slice(0, 1))
    tiny = (slice(1, 2), slice(None)) if small == "entry" else (slice(None), slice(1, 2))
    wide = lambda s: slice(s.start * g, s.stop * g) if s.start is not None else s  # noqa: E731
    for part, fd, fv in ((big, 2.0 ** 8, 2.0 ** 6), (tiny, 2.0 ** -8, 2.0 ** -2)):
        do[part[0], :, wide(part[1])] *= fd
        v[part[0], :, part[1]] *= fv
    o, lse = vg.attention(q, k, v)
    got = vg.attention_backward(do, q, k, v, o, lse)
    vg.sync_status()
    for part in (big, tiny):
        rows = lambda a: _np(a[part[0], :, wide(part[1])])  # noqa: E731
        keys = lambda a: _np(a[part[0], :, part[1]])  # noqa: E731
        args = rows(do), rows(q), keys(k), keys(v)
        ref = ot.attention_backward(*args)
        tol = ot.attention_backward_bounds(*args, U["f16"], SUM, tiny=2.0 ** -38)
        for a, r, e in zip((rows(got[0]), keys(got[1]), keys(got[2])), ref, tol):
            e = 1.01 * e + U["f16"] * np.abs(r) * 1.001 + FLOOR["f16"]
            # f16 ends at 65504, and from 65520 on (half a step of 32 further) a value rounds to infinity: some of the
            # large part's dq lie there. An infinity of the right sign is right where the bound reaches that far.
            over = np.isinf(a) & (np.sign(a) == np.sign(r)) & (np.abs(r) + e >= 65520.0)
            assert part is big or not over.any()
            _within(np.where(over, r, a), r, e)


# ───────────────────────────── shapes ─────────────────────────────

SHAPES = [
    # more entries than a warp has lanes, the keys over CTAs; lengths of 0 and 1 among them
    (40, 1, 700, 4, 1, 64, "bf16", 0, None, [(e * 97) % 701 for e in range(40)]),
    (33, 2, 1500, 1, 1, 128, "f16", 1, None, [0] * 5 + [1500, 1] + [1500 - 40 * e for e in range(26)]),
    (70, 1, 300, 2, 1, 40, "f16", 0, None, None),
    # groups of 3, 5, 6, 7 and 15 heads to a key head, keys over CTAs and not
    (2, 1, 3000, 12, 4, 128, "bf16", 0, None, [3000, 1111]), (2, 1, 2000, 5, 1, 64, "f16", 0, None, None),
    (1, 2, 1500, 14, 2, 96, "bf16", 5, None, None), (2, 3, 900, 12, 2, 64, "f16", 0, None, [900, 1]),
    (1, 1, 200, 15, 1, 72, "f16", 0, None, None), (1, 150, 150, 7, 1, 64, "bf16", 32, None, None),
]


@pytest.mark.parametrize("case", SHAPES)
def test_attention_many_entries_and_odd_groups(case):
    base.test_attention(case)


@pytest.mark.parametrize("case", SHAPES)
def test_attention_backward_many_entries_and_odd_groups(case):
    base.test_attention_backward(case)


# ───────────────────────────── rows of few keys ─────────────────────────────

@pytest.mark.parametrize("case", [(1, 1024, 1024, 8, 8, 64, "bf16", 1, None, None), (1, 1000, 1000, 2, 1, 40, "f16", 1, None, None),
                                  (3, 200, 1024, 2, 2, 128, "bf16", 0, None, [1024, 256, 129])])
def test_attention_backward_rows_of_few_keys(case):
    """Rows whose tile of 128 rows meets at most 256 keys take D from p and dp, whether or not the other rows' keys are
    split over CTAs: where p and dp leave little of dS, D from the rounded output would show."""
    b, sq, sk, hq, hkv, d, t, block, _, k_len = case
    (q, k, v, do), (q64, k64, v64, do64), kw, okw = _att_inputs(case)
    o, lse = vg.attention(q, k, v, **kw)
    dq, _, _ = vg.attention_backward(do, q, k, v, o, lse, **kw)
    vg.sync_status()
    ref = ot.attention_backward(do64, q64, k64, v64, **okw)[0]
    tol = ot.attention_backward_bounds(do64, q64, k64, v64, U[t], SUM, tiny=2.0 ** -38 if t == "f16" else 2.0 ** -100,
                                       exact_d=True, **okw)[0]
    tol = 1.01 * tol + U[t] * np.abs(ref) * 1.001 + FLOOR[t]
    got = _np(dq)
    kl = [sk] * b if k_len is None else k_len
    for e in range(b):
        if block == 0 and kl[e] > 256:
            continue
        rows = sq if block == 0 else 256 // (hq // hkv)  # (causal from position 0, heads of a group side by side)
        _within(got[e, :rows], ref[e, :rows], tol[e, :rows])
