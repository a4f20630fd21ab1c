"""Pins of the oracle's token operators (CPU only): gradients against central
differences, closed forms of the rotation, hand-written masks and empty rows."""
import numpy as np
import pytest

from oracle import tokens as ot


def _rng(seed):
    return np.random.default_rng([seed, 77])


def _differences(f, x, dirs, h=1e-5):
    """Directional derivatives of the scalar f at x by central differences."""
    return np.array([(f(x + h * d) - f(x - h * d)) / (2 * h) for d in dirs])


def test_layernorm_moments_and_gradients():
    r = _rng(0)
    x, g, b, dy = r.standard_normal((5, 7)) * 2 + 1, r.standard_normal(7), r.standard_normal(7), r.standard_normal((5, 7))
    y = ot.layernorm(x, eps=0.0)
    assert np.abs(y.mean(1)).max() < 1e-14 and np.abs((y * y).mean(1) - 1).max() < 1e-13
    dx, dg, db = ot.layernorm_backward(dy, x, g, eps=1e-3)
    dirs = r.standard_normal((6, 5, 7))
    num = _differences(lambda t: (dy * ot.layernorm(t, g, b, 1e-3)).sum(), x, dirs)
    assert np.abs(num - (dirs * dx).sum((1, 2))).max() < 1e-7
    num = _differences(lambda t: (dy * ot.layernorm(x, t, b, 1e-3)).sum(), g, dirs[:, 0])
    assert np.abs(num - dirs[:, 0] @ dg).max() < 1e-7
    num = _differences(lambda t: (dy * ot.layernorm(x, g, t, 1e-3)).sum(), b, dirs[:, 0])
    assert np.abs(num - dirs[:, 0] @ db).max() < 1e-7


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_turns_pairs_and_turns_back(interleaved):
    r = _rng(1)
    x = r.standard_normal((2, 3, 2, 10))
    pos = r.integers(0, 50, (2, 3, 2)).astype(float)
    y = ot.rope(x, pos, (2, 6), interleaved=interleaved)
    # the first pair turns by the first axis' position itself, channels 8 and 9 are copied
    ia, ib = (0, 1) if interleaved else (0, 4)
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * pos[..., 0])[..., None]
    assert np.abs(y[..., ia] - z.real).max() < 1e-14 and np.abs(y[..., ib] - z.imag).max() < 1e-14
    assert (y[..., 8:] == x[..., 8:]).all()
    # pair 3 (the third of axis 1): theta^(-4/6) of the second axis' position
    ia, ib = (6, 7) if interleaved else (3, 7)
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * pos[..., 1] * 10000.0 ** (-4 / 6))[..., None]
    assert np.abs(y[..., ia] - z.real).max() < 1e-13 and np.abs(y[..., ib] - z.imag).max() < 1e-13
    assert np.abs(ot.rope(y, pos, (2, 6), interleaved=interleaved, inverse=True) - x).max() < 1e-14
    # the inverse is the transpose: <dy, rope(x)> = <rope_inverse(dy), x>
    dy = r.standard_normal(x.shape)
    back = ot.rope(dy, pos, (2, 6), interleaved=interleaved, inverse=True)
    assert abs((dy * y).sum() - (back * x).sum()) < 1e-12


def test_seen_by_hand():
    assert ot.seen(3, 3, 0).all()
    assert (ot.seen(3, 3, 1) == np.tril(np.ones((3, 3), bool))).all()
    # two queries at positions 3, 4 of five keys, blocks of two: keys 0-3 and 0-4
    assert (ot.seen(2, 5, 2) == np.array([[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]], bool)).all()
    # more queries than keys: those at negative positions see nothing
    assert (ot.seen(4, 2, 2) == np.array([[0, 0], [0, 0], [1, 1], [1, 1]], bool)).all()


def test_attention_rows_that_see_nothing_and_single_keys():
    r = _rng(2)
    q, k, v = r.standard_normal((2, 4, 2, 8)), r.standard_normal((2, 3, 1, 8)), r.standard_normal((2, 3, 1, 8))
    o, lse = ot.attention(q, k, v, k_len=[0, 1], q_len=[4, 2])
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    assert np.abs(o[1, :2] - v[1, 0]).max() < 1e-15 and (o[1, 2:] == 0).all()
    assert np.abs(lse[1, :, :2] - np.einsum("ihd,d->hi", q[1, :2], k[1, 0, 0]) / np.sqrt(8)).max() < 1e-14
    o, lse = ot.attention(q, k, v, block=1)
    assert (o[:, 0] == 0).all() and np.isneginf(lse[:, :, 0]).all() and np.isfinite(lse[:, :, 1:]).all()


@pytest.mark.parametrize("block,q_len,k_len", [(0, None, None), (2, None, None), (3, [3, 5], [6, 2])])
def test_attention_gradients_against_differences(block, q_len, k_len):
    r = _rng(3)
    q, k, v = r.standard_normal((2, 5, 4, 8)), r.standard_normal((2, 6, 2, 8)), r.standard_normal((2, 6, 2, 8))
    do = r.standard_normal(q.shape)
    do0 = do.copy()
    if q_len is not None:
        for e, n in enumerate(q_len):
            do0[e, n:] = 0
    kw = dict(scale=0.4, q_len=q_len, k_len=k_len, block=block)
    f = lambda *a: (do0 * ot.attention(*a, **kw)[0]).sum()  # noqa: E731
    grads = ot.attention_backward(do, q, k, v, **kw)
    for i, x in enumerate((q, k, v)):
        args = [q, k, v]
        dirs = r.standard_normal((4,) + x.shape)
        num = _differences(lambda t: f(*[t if j == i else a for j, a in enumerate(args)]), x, dirs)
        assert np.abs(num - (dirs * grads[i]).sum((1, 2, 3, 4))).max() < 1e-7
