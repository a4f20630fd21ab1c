"""Refusals of the norm of query and key heads with rotary positions (CPU only):
every bad argument is answered before anything touches a GPU."""
import ctypes

import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from implicit_gemm_convolution_vae_gb300.build import build

FAKE = 1 << 24  # non-NULL, aligned, never dereferenced
MB = 1 << 20
F32, F16, BF16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    build()
    return vg.lib()


class Desc(ctypes.Structure):
    """vae_qk_norm_rope_desc as the header declares it."""
    _fields_ = [(n, ctypes.c_int) for n in ("type", "b", "s", "hq", "hk", "d")] + [("eps", ctypes.c_float)] + \
        [(n, ctypes.c_int) for n in ("pos_int", "pos_batch")] + \
        [(n + "_stride", ctypes.c_longlong * 3) for n in ("q", "k", "q_out", "k_out", "dq_out", "dk_out")]


def _three(*v):
    return (ctypes.c_longlong * 3)(*v)


def _desc(**kw):
    b, s, hq, hk, d = (kw.pop(k, v) for k, v in (("b", 2), ("s", 40), ("hq", 6), ("hk", 2), ("d", 64)))
    a = Desc(kw.pop("type", F16), b, s, hq, hk, d, kw.pop("eps", 1e-6), kw.pop("pos_int", 0), kw.pop("pos_batch", 1))
    for n, h in (("q", hq), ("q_out", hq), ("dq_out", hq), ("k", hk), ("k_out", hk), ("dk_out", hk)):
        setattr(a, n + "_stride", _three(s * h * d, h * d, d))
    for k, v in kw.items():
        setattr(a, k, _three(*v))
    return a


def _plan(L, dims=(16, 24, 24), inter=1):
    p = vg._RopePlan()
    assert L.vae_rope_plan_init(ctypes.byref(p), len(dims), (ctypes.c_int * len(dims))(*dims), 10000.0, inter) == 0
    return p


def test_binding_packs_the_desc_as_declared(L):
    a = Desc(2, 3, 4, 5, 6, 7, 0.5, 1, 3)
    for i, n in enumerate(("q", "k", "q_out", "k_out", "dq_out", "dk_out")):
        setattr(a, n + "_stride", _three(*[(i * 3 + j + 1) << 33 for j in range(3)]))
    assert bytes(a) == vg._QK_DESC.pack(2, 3, 4, 5, 6, 7, 0.5, True, 3, *[(i + 1) << 33 for i in range(18)])


def test_forward_refusals(L):
    plan = _plan(L)
    ok = dict(q=FAKE, k=FAKE + MB, gq=FAKE + 2 * MB, gk=FAKE + 3 * MB, pos=FAKE + 4 * MB, plan=ctypes.byref(plan),
              qo=FAKE + 5 * MB, ko=FAKE + 6 * MB)

    def rc(desc=None, **kw):
        a = {**ok, **kw}
        return L.vae_qk_norm_rope(ctypes.byref(desc if desc is not None else _desc()), a["q"], a["k"], a["gq"], a["gk"],
                                  a["pos"], a["plan"], a["qo"], a["ko"], None)

    assert L.vae_qk_norm_rope(None, FAKE, FAKE, None, None, None, None, FAKE, FAKE, None) == -1
    for k in ("q", "k", "qo", "ko", "pos", "plan"):
        assert rc(**{k: None}) == -1
    assert "together" in vg.last_error()
    assert rc(_desc(type=3)) == -1 and rc(plan=ctypes.byref(vg._RopePlan())) == -1
    for n in ("b", "s", "hq", "hk", "d"):
        assert rc(_desc(**{n: 0})) == -2 and rc(_desc(**{n: -3})) == -2
    assert rc(_desc(d=257)) == -2 and rc(_desc(d=62)) == -2 and "62" in vg.last_error()
    assert rc(_desc(b=1 << 16, s=1 << 15)) == -2 and rc(_desc(hq=1 << 19, hk=1 << 19)) == -2
    for eps in (0.0, -1.0, NAN, INF):
        assert rc(_desc(eps=eps)) == -1
    assert rc(_desc(pos_batch=3)) == -2 and rc(_desc(pos_batch=0)) == -2
    assert rc(_desc(q_stride=(15360, -384, 64))) == -2 and rc(_desc(k_out_stride=(0, 128, 64))) == -2
    assert rc(_desc(q_out_stride=(15360, 384, 32))) == -2 and "lie in one another" in vg.last_error()
    assert rc(q=FAKE + 1) == -3 and rc(ko=FAKE + 6 * MB + 1) == -3 and rc(pos=FAKE + 2) == -3 and rc(gq=FAKE + 2) == -3
    # what is written and what is read
    assert rc(qo=FAKE + 128) == -1 and rc(qo=FAKE + MB) == -1 and rc(ko=FAKE) == -1
    assert rc(qo=FAKE + 6 * MB) == -1 and rc(qo=FAKE + 2 * MB) == -1 and rc(ko=FAKE + 4 * MB + 64) == -1
    assert rc(_desc(q_out_stride=(15360 * 2, 384, 64)), qo=FAKE) == -1 and "same strides" in vg.last_error()


def test_backward_refusals(L):
    plan = _plan(L)
    ws = L.vae_qk_norm_rope_backward_workspace_bytes(ctypes.byref(_desc()))
    assert ws >= 2 * 64 * 4
    assert L.vae_qk_norm_rope_backward_workspace_bytes(None) == 0
    assert L.vae_qk_norm_rope_backward_workspace_bytes(ctypes.byref(_desc(d=300))) == 0
    at = {n: FAKE + i * MB for i, n in enumerate(("gq", "gk", "q", "k", "wq", "wk", "pos", "dq", "dk", "dwq", "dwk", "ws"))}
    ok = dict(at, plan=ctypes.byref(plan), n=ws)

    def rc(desc=None, **kw):
        a = {**ok, **kw}
        return L.vae_qk_norm_rope_backward(ctypes.byref(desc if desc is not None else _desc()), a["gq"], a["gk"], a["q"],
                                           a["k"], a["wq"], a["wk"], a["pos"], a["plan"], a["dq"], a["dk"], a["dwq"],
                                           a["dwk"], a["ws"], a["n"], None)

    for k in ("gq", "gk", "q", "k", "dq", "dk", "dwq", "dwk", "pos", "plan", "ws"):
        assert rc(**{k: None}) == -1, k
    assert rc(n=ws - 1) == -4 and rc(ws=at["ws"] + 8) == -3
    assert rc(dq=at["dq"] + 1) == -3 and rc(dwk=at["dwk"] + 2) == -3
    assert rc(_desc(dq_out_stride=(15360, -1, 64))) == -2
    assert rc(dq=at["k"]) == -1 and rc(dq=at["gk"]) == -1 and rc(dk=at["gq"]) == -1 and rc(dq=at["dk"]) == -1
    assert rc(dq=at["gq"] + 128) == -1 and rc(dwq=at["dwk"]) == -1 and rc(dwq=at["wq"]) == -1 and rc(ws=at["q"]) == -1
    assert rc(dwk=at["pos"]) == -1 and rc(ws=at["dk"]) == -1
    assert rc(_desc(q_out_stride=(15360 * 2, 384, 64)), dq=at["gq"]) == -1 and "same strides" in vg.last_error()


def test_workspace_is_a_function_of_the_sizes(L):
    f = vg.qk_norm_rope_backward_workspace_bytes
    assert f(1, 1, 1, 1, 128) == 2 * 128 * 4
    assert f(4, 1 << 20, 16, 4, 128) == f(1, 1 << 20, 3, 1, 128)
    with pytest.raises(vg.VaeError):
        f(1, 1 << 40, 1, 1, 128)


def test_binding_refuses_what_is_no_cuda_tensor(L):
    import torch
    x = torch.zeros(1, 2, 3, 8)
    with pytest.raises(vg.VaeError, match="CUDA"):
        vg.qk_norm_rope(x, x)
    with pytest.raises(vg.VaeError, match="needed"):
        vg.qk_norm_rope(x, None)
    with pytest.raises(vg.VaeError, match="needed"):
        vg.qk_norm_rope_backward(x, x, None, x)
