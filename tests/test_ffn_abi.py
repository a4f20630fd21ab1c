"""Refusals of the gated feed-forward block (CPU only): every bad argument is
answered before anything touches a GPU."""
import ctypes

import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from implicit_gemm_convolution_vae_gb300.build import build

FAKE = 1 << 24  # non-NULL, aligned, never dereferenced
MB = 1 << 20
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    build()
    return vg.lib()


class Desc(ctypes.Structure):
    """vae_gated_ffn_desc as the header declares it."""
    _fields_ = [(n, ctypes.c_int) for n in ("type", "m", "c", "f", "activation", "y_type", "save", "dw_type")]


def _desc(**kw):
    return ctypes.byref(Desc(*({**dict(type=F16, m=40, c=64, f=128, activation=0, y_type=F16, save=0, dw_type=F16), **kw}.values())))


def test_binding_packs_the_desc_as_declared():
    assert bytes(Desc(1, 2, 3, 4, 5, 6, 7, 8)) == vg._FFN_DESC.pack(1, 2, 3, 4, 5, 6, 7, 8)


BAD_SHAPES = [dict(m=0), dict(m=-1), dict(m=(1 << 24) + 1), dict(c=0), dict(c=60), dict(c=4), dict(c=16392), dict(f=0), dict(f=-8),
              dict(f=100), dict(f=65544)]


def test_forward_refusals(L):
    names = ("x", "wg", "wu", "wd", "res", "y", "gate", "up", "hidden", "ws")
    at = {n: FAKE + i * MB for i, n in enumerate(names)}
    at.update(res=None, gate=None, up=None, hidden=None)
    need = L.vae_gated_ffn_workspace_bytes(_desc())

    def rc(desc=None, n=None, **kw):
        a = {**at, **kw}
        return L.vae_gated_ffn(desc if desc is not None else _desc(), *[a[k] for k in names], need if n is None else n, None)

    assert need >= 40 * 128 * 2
    assert L.vae_gated_ffn_workspace_bytes(None) == 0 and rc(n=need - 1) == -4
    assert L.vae_gated_ffn(None, *[at[k] for k in names], need, None) == -1
    for k in ("x", "wg", "wu", "wd", "y", "ws"):
        assert rc(**{k: None}) == -1, k
    for bad in BAD_SHAPES:
        assert rc(_desc(**bad)) == -2 and L.vae_gated_ffn_workspace_bytes(_desc(**bad)) == 0
    assert rc(_desc(type=F32)) == -1 and rc(_desc(type=3)) == -1 and rc(_desc(activation=3)) == -1 and rc(_desc(activation=-1)) == -1
    assert rc(_desc(y_type=BF16)) == -1 and rc(res=FAKE + 20 * MB) == -1 and "residual" in vg.last_error()
    assert rc(gate=FAKE + 20 * MB) == -1 and rc(_desc(save=1)) == -1
    save = dict(gate=FAKE + 20 * MB, up=FAKE + 21 * MB, hidden=FAKE + 22 * MB)
    assert rc(_desc(save=1), **{**save, "up": None}) == -1
    for k in ("x", "wg", "wu", "wd", "y", "ws"):
        assert rc(**{k: at[k] + 8}) == -3, k
    # what is written lies apart
    for k in ("x", "wg", "wu", "wd", "ws"):
        assert rc(y=at[k]) == -1 and "overlap" in vg.last_error()
    assert rc(y=at["x"] + 16) == -1 and rc(ws=at["wd"] + 64) == -1
    assert rc(_desc(save=1), **{**save, "gate": at["x"]}) == -1 and rc(_desc(save=1), **{**save, "gate": save["up"] + 16}) == -1
    assert rc(_desc(y_type=F32), res=at["y"] + 16) == -1 and rc(_desc(y_type=F32), res=at["ws"]) == -1


def test_backward_refusals(L):
    names = ("dy", "x", "wg", "wu", "wd", "gate", "up", "hidden", "dx", "dwg", "dwu", "dwd", "ws")
    at = {n: FAKE + i * MB for i, n in enumerate(names)}
    need = L.vae_gated_ffn_backward_workspace_bytes(_desc())

    def rc(desc=None, n=None, **kw):
        a = {**at, **kw}
        return L.vae_gated_ffn_backward(desc if desc is not None else _desc(), *[a[k] for k in names], need if n is None else n, None)

    assert need >= 2 * 40 * 128 * 2
    assert rc(n=need - 1) == -4
    assert L.vae_gated_ffn_backward(None, *[at[k] for k in names], need, None) == -1
    for k in names:
        assert rc(**{k: None}) == -1, k
    assert rc(dwg=None, dwu=None) == -1 and "together" in vg.last_error()
    for bad in BAD_SHAPES:
        assert rc(_desc(**bad)) == -2 and L.vae_gated_ffn_backward_workspace_bytes(_desc(**bad)) == 0
    assert rc(_desc(type=F32)) == -1 and rc(_desc(dw_type=BF16)) == -1 and rc(_desc(activation=9)) == -1
    for k in names:
        assert rc(**{k: at[k] + 8}) == -3, k
    for w in ("dx", "dwg", "dwu", "dwd", "ws"):
        for k in names:
            if k != w:
                assert rc(**{w: at[k]}) == -1, (w, k)
    assert rc(_desc(dw_type=F32), dwd=at["dwu"] + 64 * 128 * 4 - 16) == -1


def test_binding_refuses(L):
    import torch
    x, w, d = torch.zeros(2, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(vg.VaeError, match="CUDA"):
        vg.gated_ffn(x, w, w, d)
    with pytest.raises(vg.VaeError, match="needed"):
        vg.gated_ffn(x, w, None, d)
    with pytest.raises(vg.VaeError, match="needed"):
        vg.gated_ffn_backward(x, x, w, w, d, (w, None, w))
    with pytest.raises(vg.VaeError, match="2\\^31"):
        vg.gated_ffn_workspace_bytes(1 << 40, 8, 8)
    assert vg.gated_ffn_workspace_bytes(100, 64, 128, save=True) == 0
