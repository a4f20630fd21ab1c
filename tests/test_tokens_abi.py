"""Refusals of the token operators (CPU only): every bad argument is answered
with its status code before anything touches a GPU, in the C ABI and in the
binding, and the workspace sizes are plain functions of the shape."""
import ctypes

import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from implicit_gemm_convolution_vae_gb300.build import build

FAKE = 1 << 20  # a non-NULL, aligned address never dereferenced: validation fails first
F32, F16, BF16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    build()
    return vg.lib()


def test_layernorm_refusals(L):
    ok = dict(x=FAKE, xt=F32, m=4, c=64, g=FAKE, b=FAKE, eps=1e-6, y=FAKE + 65536, yt=F16)

    def rc(**kw):
        a = {**ok, **kw}
        return L.vae_layernorm(a["x"], a["xt"], a["m"], a["c"], a["g"], a["b"], a["eps"], a["y"], a["yt"], None)

    assert rc(x=None) == -1 and rc(y=None) == -1
    assert rc(xt=3) == -1 and rc(yt=-1) == -1
    assert rc(m=0) == -2 and rc(c=0) == -2 and rc(c=16385) == -2
    assert rc(eps=-1.0) == -1 and rc(eps=NAN) == -1 and rc(eps=INF) == -1
    assert rc(y=FAKE) == -1 and "in place" in vg.last_error()
    assert rc(x=FAKE + 4) == -3 and rc(y=FAKE + 2) == -3 and rc(g=FAKE + 4) == -3
    assert rc(c=63, x=FAKE + 2) == -3 and rc(c=63, y=FAKE + 65537) == -3 and rc(c=63, b=FAKE + 2) == -3


def test_layernorm_backward_refusals(L):
    ws = L.vae_layernorm_backward_workspace_bytes(100, 64)
    assert ws > 0
    assert L.vae_layernorm_backward_workspace_bytes(0, 64) == 0
    assert L.vae_layernorm_backward_workspace_bytes(4, 16385) == 0
    ok = dict(dy=FAKE, dyt=F16, x=FAKE, xt=F32, m=100, c=64, g=FAKE, eps=1e-6, dx=FAKE, dg=FAKE, db=FAKE, w=FAKE, n=ws)

    def rc(**kw):
        a = {**ok, **kw}
        return L.vae_layernorm_backward(a["dy"], a["dyt"], a["x"], a["xt"], a["m"], a["c"], a["g"], a["eps"], a["dx"],
                                        a["dg"], a["db"], a["w"], a["n"], None)

    assert rc(dy=None) == -1 and rc(x=None) == -1 and rc(dx=None) == -1
    assert rc(dyt=7) == -1 and rc(m=-1) == -2 and rc(c=20000) == -2
    assert rc(dg=None) == -1 and "together" in vg.last_error()
    assert rc(dx=FAKE) == -1 and "dx over dy" in vg.last_error()
    assert rc(dx=FAKE + 4096, w=None) == -1
    assert rc(dx=FAKE + 4096, n=ws - 1) == -4
    assert rc(dx=FAKE + 8) == -3


def _plan(L, dims=(16, 24, 24), theta=10000.0, inter=1):
    p = vg._RopePlan()
    return L.vae_rope_plan_init(ctypes.byref(p), len(dims), (ctypes.c_int * max(1, len(dims)))(*dims), theta, inter), p


def test_rope_refusals(L):
    assert _plan(L)[0] == 0
    assert _plan(L, dims=())[0] == -2 and _plan(L, dims=(2,) * 5)[0] == -2
    assert _plan(L, dims=(3,))[0] == -2 and _plan(L, dims=(-2, 4))[0] == -2
    assert _plan(L, dims=(0, 0))[0] == -2 and _plan(L, dims=(256, 2))[0] == -2
    assert _plan(L, theta=0.5)[0] == -1 and _plan(L, theta=NAN)[0] == -1 and _plan(L, theta=INF)[0] == -1
    assert L.vae_rope_plan_init(None, 1, (ctypes.c_int * 1)(2), 10.0, 1) == -1
    rc0, plan = _plan(L)
    st = lambda *v: (ctypes.c_longlong * 3)(*v)  # noqa: E731
    ok = dict(x=FAKE, t=F16, b=2, s=5, h=3, d=64, xs=st(960, 192, 64), pos=FAKE, pi=0, pb=1, plan=ctypes.byref(plan),
              y=FAKE + (1 << 20), ys=st(960, 192, 64))

    def rc(**kw):
        a = {**ok, **kw}
        return L.vae_rope(a["x"], a["t"], a["b"], a["s"], a["h"], a["d"], a["xs"], a["pos"], a["pi"], a["pb"], a["plan"],
                          0, a["y"], a["ys"], None)

    for k in ("x", "y", "pos", "plan", "xs", "ys"):
        assert rc(**{k: None}) == -1
    assert rc(t=3) == -1 and rc(plan=ctypes.byref(vg._RopePlan())) == -1
    assert rc(b=0) == -2 and rc(s=0) == -2 and rc(h=0) == -2 and rc(d=62) == -2 and rc(d=258) == -2
    assert rc(b=1 << 16, s=1 << 15) == -2 and rc(h=1 << 20) == -2
    assert rc(pb=3) == -2 and rc(pb=0) == -2
    assert rc(xs=st(960, -192, 64)) == -2 and rc(ys=st(0, 192, 64)) == -2
    assert rc(y=FAKE, ys=st(960, 192, 128)) == -1
    assert rc(x=FAKE + 1) == -3 and rc(pos=FAKE + 2) == -3


class AttentionDesc(ctypes.Structure):
    """vae_attention_desc as the header declares it."""
    _fields_ = [(n, ctypes.c_int) for n in ("type", "b", "sq", "sk", "hq", "hkv", "d")] + \
        [("scale", ctypes.c_float), ("block", ctypes.c_int), ("fill", ctypes.c_int), ("q_len", ctypes.c_void_p), ("k_len", ctypes.c_void_p)] + \
        [(n + "_stride", ctypes.c_longlong * 3) for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")]


def test_binding_packs_the_desc_as_declared(L):
    a = AttentionDesc(2, 3, 4, 5, 6, 7, 8, 0.5, 9, 1, 1 << 40, 1 << 41)
    for i, n in enumerate(("q", "k", "v", "o", "do", "dq", "dk", "dv")):
        setattr(a, n + "_stride", (ctypes.c_longlong * 3)(*[(i * 3 + j + 1) << 33 for j in range(3)]))
    assert bytes(a) == vg._DESC.pack(2, 3, 4, 5, 6, 7, 8, 0.5, 9, True, 1 << 40, 1 << 41, *[(i + 1) << 33 for i in range(24)])


def _dense(b, n, h, d):
    return (ctypes.c_longlong * 3)(n * h * d, h * d, d)


def _desc(**kw):
    b, sq, sk, hq, hkv, d = (kw.pop(k, v) for k, v in (("b", 2), ("sq", 40), ("sk", 50), ("hq", 6), ("hkv", 3), ("d", 64)))
    a = AttentionDesc(kw.pop("type", F16), b, sq, sk, hq, hkv, d, kw.pop("scale", 0.125), kw.pop("block", 0))
    for n in ("q", "o", "do", "dq"):
        setattr(a, n + "_stride", _dense(b, sq, hq, d))
    for n in ("k", "v", "dk", "dv"):
        setattr(a, n + "_stride", _dense(b, sk, hkv, d))
    for k, v in kw.items():
        setattr(a, k, (ctypes.c_longlong * 3)(*v))
    return a


P5 = [FAKE + i * 65536 for i in range(5)]
P10 = [FAKE + i * 65536 for i in range(10)]
BAD = [(dict(type=F32), -1), (dict(type=9), -1), (dict(b=0), -2), (dict(sq=0), -2), (dict(sk=0), -2), (dict(hq=0), -2),
       (dict(hkv=0), -2), (dict(hq=7), -2), (dict(d=0), -2), (dict(d=12), -2), (dict(d=136), -2), (dict(scale=0.0), -1),
       (dict(scale=-1.0), -1), (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(block=-1), -1),
       (dict(q_stride=(15360, 384, 60)), -2), (dict(k_stride=(9600, 192, 0)), -2), (dict(v_stride=(9600, -192, 64)), -2),
       (dict(o_stride=(0, 384, 64)), -2), (dict(o_stride=(15360, 384, 56)), -2), (dict(b=1 << 12, sq=1 << 20), -2)]


@pytest.mark.parametrize("bad,code", BAD)
def test_attention_refuses_bad_descs(L, bad, code):
    a = ctypes.byref(_desc(**bad))
    assert L.vae_attention_backward_workspace_bytes(a) == 0
    assert L.vae_attention(a, *P5, FAKE, 1 << 40, None) == code
    assert L.vae_attention_backward(a, *P10, 1 << 40, None) == code


def test_attention_refuses_bad_pointers_and_workspaces(L):
    a = ctypes.byref(_desc())
    assert L.vae_attention(None, *P5, FAKE, 1 << 40, None) == -1
    for i in range(5):
        p = list(P5)
        p[i] = None
        assert L.vae_attention(a, *p, FAKE, 1 << 40, None) == -1
        p[i] = FAKE + 8
        assert L.vae_attention(a, *p, FAKE, 1 << 40, None) == -3
    for i in range(3):  # o over q, k or v
        p = list(P5)
        p[3] = p[i]
        assert L.vae_attention(a, *p, FAKE, 1 << 40, None) == -1
        assert "may not be" in vg.last_error()
    assert L.vae_attention_backward(None, *P10, 1 << 40, None) == -1
    for i in range(10):
        p = list(P10)
        p[i] = None
        assert L.vae_attention_backward(a, *p, 1 << 40, None) == -1
        p[i] = FAKE + 8
        assert L.vae_attention_backward(a, *p, 1 << 40, None) == -3
    for i in (6, 7, 8):  # a gradient over an input, or over another
        for j in (0, 1, 2, 3, 4, 6 + (i - 5) % 3):
            p = list(P10)
            p[i] = p[j]
            assert L.vae_attention_backward(a, *p, 1 << 40, None) == -1
    n = L.vae_attention_backward_workspace_bytes(a)
    assert n > 0 and n % 16 == 0
    assert L.vae_attention_backward(a, *P10, n - 1, None) == -4
    for bad in (dict(do_stride=(15360, 384, 4)), dict(dq_stride=(15360, 0, 64)), dict(dk_stride=(1, 192, 64)),
                dict(dv_stride=(9600, 192, -64)), dict(dq_stride=(15360, 384, 32))):
        assert L.vae_attention_backward(ctypes.byref(_desc(**bad)), *P10, 1 << 40, None) == -2


def test_workspace_sizes_follow_the_shape(L):
    assert vg.attention_backward_workspace_bytes(2, 100, 100, 4, 2, 64) > 0
    assert vg.attention_workspace_bytes(1, 1, 1, 1, 1, 8) == vg.attention_workspace_bytes(1, 1, 1, 1, 1, 8)
    assert vg.layernorm_backward_workspace_bytes(1 << 20, 1152) == vg.layernorm_backward_workspace_bytes(1 << 21, 1152)


def test_binding_refuses_cpu_tensors_and_wrong_shapes(L):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(vg.VaeError, match="CUDA tensor"):
        vg.layernorm(x)
    with pytest.raises(vg.VaeError, match="is needed"):
        vg.layernorm(None)
    with pytest.raises(vg.VaeError, match="CUDA tensor"):
        vg.layernorm_backward(x, x)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.float16)
    with pytest.raises(vg.VaeError, match="CUDA tensor"):
        vg.attention(q, q, q)
    with pytest.raises(vg.VaeError, match="is needed"):
        vg.attention_backward(None, q, q, q, q, None)
    with pytest.raises(vg.VaeError, match="CUDA tensor"):
        vg.rope(q, torch.zeros(4, 3), vg.RopePlan((16, 24, 24)))
    with pytest.raises(vg.VaeError, match="even"):
        vg.RopePlan((3, 5))


def test_no_cpu_fallback_without_a_gpu(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.vae_layernorm(FAKE, F32, 4, 64, None, None, 1e-6, FAKE, F32, None) in (-5, -7)
    n = 1 << 40
    assert L.vae_attention(ctypes.byref(_desc()), *P5, FAKE, n, None) in (-5, -7)
    assert L.vae_attention_backward(ctypes.byref(_desc()), *P10, n, None) in (-5, -7)
