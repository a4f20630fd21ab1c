"""Pins of the float64 oracle of the heads' norm with rotary positions and of the gated
feed-forward block (CPU only): closed forms, and gradients against differences."""
import numpy as np
import pytest

from oracle import tokens as ot
from vae_inputs import rng_for


def _r(name, *shape):
    return rng_for(40, "pin." + name).standard_normal(shape)


def test_qk_norm_of_known_rows():
    x = np.array([3.0, -4.0, 0.0, 0.0]).reshape(1, 1, 1, 4)
    # mean square 25 / 4: the norm divides by 2.5
    assert np.allclose(ot.qk_norm_rope(x, eps=0.0).ravel(), [1.2, -1.6, 0.0, 0.0])
    # position pi / 2 of the first pair's angle 1: (a, b) -> (-b, a); the second pair's angle is theta^(-1/2) times it
    y = ot.qk_norm_rope(x, np.array([2.0, 1.0, 1.0, 1.0]), np.array([[np.pi / 2]]), (4,), 1e30, True, eps=0.0).ravel()
    assert np.allclose(y, [1.6, 2.4, 0.0, 0.0])


def test_qk_norm_keeps_the_size_of_a_row():
    x = _r("size", 2, 3, 4, 32)
    y = ot.qk_norm_rope(x, None, np.arange(6.0).reshape(2, 3, 1), (20,), eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)


@pytest.mark.parametrize("inter", [True, False])
def test_qk_norm_gradient_against_differences(inter):
    x, g, w = _r("x", 2, 3, 2, 12), 1.0 + 0.2 * _r("g", 12), _r("w", 2, 3, 2, 12)
    pos, axes = np.arange(6.0).reshape(3, 2), (4, 6)
    f = lambda x, g: (w * ot.qk_norm_rope(x, g, pos, axes, 100.0, inter, 1e-3)).sum()  # noqa: E731
    dx, dg = ot.qk_norm_rope_backward(w, x, g, pos, axes, 100.0, inter, 1e-3)
    for i in range(5):
        vx, vg = _r(f"vx{i}", *x.shape), _r(f"vg{i}", 12)
        h = 1e-5
        assert abs((f(x + h * vx, g) - f(x - h * vx, g)) / (2 * h) - (dx * vx).sum()) < 1e-7
        assert abs((f(x, g + h * vg) - f(x, g - h * vg)) / (2 * h) - (dg * vg).sum()) < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_activations(kind):
    g = np.linspace(-6.0, 6.0, 1201)
    v, d = ot.activation(g, kind)
    assert v[600] == 0.0 and abs(d[600] - 0.5) < 1e-15
    assert np.allclose(v - ot.activation(-g, kind)[0], g)  # act(g) - act(-g) = g for all three
    h = 1e-5
    assert np.abs((ot.activation(g + h, kind)[0] - ot.activation(g - h, kind)[0]) / (2 * h) - d).max() < 1e-9
    at1 = {"silu": 0.7310585786300049, "gelu": 0.8413447460685429, "gelu_tanh": 0.8411919906082768}[kind]
    assert abs(ot.activation(1.0, kind)[0] - at1) < 1e-12


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_gated_ffn_gradient_against_differences(kind):
    x, wg, wu, wd, w = _r("fx", 5, 6), _r("fg", 7, 6), _r("fu", 7, 6), _r("fd", 6, 7), _r("fw", 5, 6)
    args = [x, wg, wu, wd]
    f = lambda *a: (w * ot.gated_ffn(*a, kind)[0]).sum()  # noqa: E731
    _, gate, up, hidden = ot.gated_ffn(*args, kind)
    grads = ot.gated_ffn_backward(w, *args, gate, up, hidden, kind)[:4]
    h = 1e-5
    for i, g in enumerate(grads):
        v = _r(f"fv{i}", *args[i].shape)
        up_, down = list(args), list(args)
        up_[i], down[i] = args[i] + h * v, args[i] - h * v
        assert abs((f(*up_) - f(*down)) / (2 * h) - (g * v).sum()) < 1e-6
