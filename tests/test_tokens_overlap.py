"""What is written lies apart from what is read (CPU only): the token operators
refuse tensors that share memory, and views that lie in one another without
meeting pass. The search behind it against every byte of small tensors."""
import ctypes
import os
import random
import subprocess

import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from implicit_gemm_convolution_vae_gb300.build import CSRC, build
from test_tokens_abi import BF16, F16, F32, FAKE, AttentionDesc, _plan

X = FAKE * 16  # where the tensors lie
NO_GPU = (-5, -7)  # the arguments were taken, and no device was found


@pytest.fixture(scope="module")
def L():
    build()
    return vg.lib()


@pytest.fixture(scope="module")
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these addresses are not real")


# ───────────────────────────── the search ─────────────────────────────

PROGRAM = r"""
#include <cstdio>
#include "vae_overlap.h"
int main() {
    long long p[2], s[2][3];
    int n[2][3], d[2];
    while (true) {
        for (int i = 0; i < 2; ++i)
            if (scanf("%lld %lld %lld %lld %d %d %d %d", &p[i], &s[i][0], &s[i][1], &s[i][2], &n[i][0], &n[i][1], &n[i][2], &d[i]) != 8) return 0;
        vae::Extent e[2];
        for (int i = 0; i < 2; ++i) e[i] = vae::extent_tokens(reinterpret_cast<const void*>(p[i]), s[i], n[i][0], n[i][1], n[i][2], d[i], 2);
        printf("%d %d\n", vae::extents_meet(e[0], e[1]), vae::extent_folds(e[0]));
    }
}
"""


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    """meet and fold of many pairs of tensors (address, strides, sizes, channels; two bytes an element)."""
    tmp = tmp_path_factory.mktemp("overlap")
    src, exe = tmp / "overlap.cpp", tmp / "overlap"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True)

    def answers(pairs):
        text = "\n".join(" ".join(str(v) for v in (t[0], *t[1], *t[2], t[3])) for pair in pairs for t in pair)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [(bool(int(a)), bool(int(b))) for a, b in zip(out[::2], out[1::2])]
    return answers


def _runs(t):
    p, st, n, d = t
    return [p + 2 * (i * st[0] + j * st[1] + k * st[2]) for i in range(n[0]) for j in range(n[1]) for k in range(n[2])]


def _bytes(t):
    return [a + x for a in _runs(t) for x in range(2 * t[3])]


def test_search_against_every_byte(search):
    rng = random.Random(5)
    pairs = []
    for _ in range(6000):
        def tensor():
            n = [rng.choice((1, 1, 2, 3, 4)) for _ in range(3)]
            d = rng.choice((1, 2, 4))
            kind = rng.random()
            if kind < 0.5:  # nested strides in some order, with or without gaps
                st, inner = [0, 0, 0], d
                for k in rng.sample(range(3), 3):
                    st[k] = inner + rng.choice((0, 0, 1, d, inner))
                    inner = st[k] * (n[k] - 1) + inner
            else:
                st = [rng.randint(0, 24) for _ in range(3)]
            return (4096 + 2 * rng.randint(0, 40), tuple(st), tuple(n), d)
        a = tensor()
        # often the same strides, a few elements further: parts of one projection
        b = (a[0] + 2 * rng.randint(-12, 12), a[1], tensor()[2], rng.choice((1, 2, 4))) if rng.random() < 0.5 else tensor()
        pairs.append((a, b))
    seen = set()
    for (a, b), (meet, fold) in zip(pairs, search(pairs)):
        ba, bb = _bytes(a), _bytes(b)
        assert meet == bool(set(ba) & set(bb)), (a, b)
        assert fold == (len(set(ba)) < len(ba)), a
        seen.add((meet, fold))
    assert len(seen) == 4


def test_search_of_large_layouts(search):
    """Parts of joint projections, heads before tokens, offsets past 32 bits, strides and sizes whose product passes 64."""
    base = 1 << 40
    b, s, h, d = 4, 16384, 16, 128
    joint = lambda i, heads: (base + 2 * i * d, (s * 3 * h * d, 3 * h * d, d), (b, s, heads), d)  # noqa: E731
    swapped = (base, (s * h * d, d, s * d), (b, s, h), d)
    vast = (base, (1 << 62, 64, 8), (4, 1 << 30, 4), 8)  # heads 0 .. 3 of eight places
    folded = (base, (1 << 38, 1 << 37, 8), (1 << 30, 1 << 30, 4), 8)  # (1, 0) lies on (0, 2)
    pairs = [(joint(0, h), joint(h, h)), (joint(h, h), joint(2 * h, h)), (joint(0, h + 1), joint(h, h)),
             (swapped, (base + 2 * b * s * h * d, *swapped[1:])), (swapped, (base + 2 * (b * s * h * d - 1), *swapped[1:])),
             (swapped, (base, (s * h * d, h * d, d), (b, s, h), d)), (vast, (base + 64, *vast[1:])), (vast, (base + 48, *vast[1:])),
             (folded, (base + 48, *folded[1:]))]
    answers = search(pairs)
    assert [m for m, _ in answers] == [False, False, True, False, True, True, False, True, True]
    assert [f for _, f in answers] == [False] * 8 + [True]


# ───────────────────────────── layer norm ─────────────────────────────

M, C = 100, 64


def test_layernorm_refuses_shared_memory(L):
    nb = M * C * 4

    def rc(y, x=X, g=X + 10 * nb, b=X + 11 * nb):
        return L.vae_layernorm(x, F32, M, C, g, b, 1e-6, y, F32, None)

    for y in (X + 16, X - 16, X + nb - 16, X - nb + 16, X + C * 4, X + 10 * nb, X + 10 * nb - nb + 16, X + 11 * nb + 16):
        assert rc(y) == -1 and "overlap" in vg.last_error(), y
    half = L.vae_layernorm(X, F32, M, C, None, None, 1e-6, X + 16, F16, None)
    assert half == -1 and "overlap" in vg.last_error()


def test_layernorm_takes_neighbours_and_in_place(L, no_gpu):
    nb = M * C * 4
    for y in (X, X + nb, X - nb, X + 10 * nb - nb, X + 11 * nb + C * 4):
        assert L.vae_layernorm(X, F32, M, C, X + 10 * nb, X + 11 * nb, 1e-6, y, F32, None) in NO_GPU


def _ln_backward(L, **kw):
    nb, ws = M * C * 4, L.vae_layernorm_backward_workspace_bytes(M, C)
    a = {**dict(dy=X, x=X + nb, g=X + 2 * nb, dx=X + 3 * nb, dg=X + 4 * nb, db=X + 5 * nb, w=X + 16 * nb), **kw}
    return L.vae_layernorm_backward(a["dy"], F32, a["x"], F32, M, C, a["g"], 1e-6, a["dx"], a["dg"], a["db"], a["w"], ws, None)


def test_layernorm_backward_refuses_shared_memory(L):
    nb, ws = M * C * 4, L.vae_layernorm_backward_workspace_bytes(M, C)
    bad = [dict(dx=X + 16), dict(dx=X + nb + 16), dict(dx=X + 2 * nb - 16), dict(dx=X + 2 * nb), dict(dg=X + 3 * nb),
           dict(db=X + 4 * nb - 16), dict(dg=X + 5 * nb + 240), dict(db=X + 4 * nb), dict(w=X + 3 * nb + 32), dict(w=X - ws + 16),
           dict(w=X + 4 * nb), dict(w=X + 5 * nb - ws + 16), dict(w=X + 2 * nb + 128), dict(w=X + nb)]
    for kw in bad:
        assert _ln_backward(L, **kw) == -1 and "overlap" in vg.last_error(), kw


def test_layernorm_backward_takes_neighbours_and_in_place(L, no_gpu):
    nb, ws = M * C * 4, L.vae_layernorm_backward_workspace_bytes(M, C)
    good = [{}, dict(dx=X), dict(dx=X + nb), dict(w=X - ws), dict(dg=X + 4 * nb, db=X + 4 * nb + C * 4), dict(dg=X + 2 * nb),
            dict(dy=X, x=X), dict(dx=X, x=X), dict(dg=None, db=None, w=None)]
    for kw in good:
        assert _ln_backward(L, **kw) in NO_GPU, (kw, vg.last_error())


# ───────────────────────────── rotary positions ─────────────────────────────

def _rope(L, x, xs, y, ys, pos=X * 8, b=2, s=5, h=3, d=64):
    st = lambda v: (ctypes.c_longlong * 3)(*v)  # noqa: E731
    return L.vae_rope(x, F16, b, s, h, d, st(xs), pos, 0, 1, ctypes.byref(_plan(L)[1]), 0, y, st(ys), None)


ROW = (5 * 8 * 64, 8 * 64, 64)  # heads 0 .. 2 of eight


def test_rope_refuses_shared_memory(L):
    for y, ys in ((X + 2, ROW), (X - 2, ROW), (X + 2 * 128, ROW), (X + 2 * 8 * 64, ROW), (X, (ROW[0], ROW[1], 128)),
                  (X + 2 * 64, (960, 192, 64))):
        assert _rope(L, X, ROW, y, ys) == -1, (y, ys)
    assert _rope(L, X, ROW, X * 8 + 32, ROW) == -1 and "overlap" in vg.last_error()
    # rows of y in one another
    for ys in ((960, 192, 32), (960, 64, 64), (192, 192, 64), (960, 100, 64)):
        assert _rope(L, X, ROW, X * 2, ys) == -2 and "row" in vg.last_error(), ys


def test_rope_takes_parts_of_a_projection_and_broadcasts(L, no_gpu):
    assert _rope(L, X, ROW, X, ROW) in NO_GPU
    for k in (3, 4, 5):  # the heads behind
        assert _rope(L, X, ROW, X + 2 * 64 * k, ROW) in NO_GPU
    assert _rope(L, X, (0, 192, 64), X * 2, (960, 192, 64)) in NO_GPU
    assert _rope(L, X, ROW, X * 2, (64, 128, 640)) in NO_GPU  # batch inside tokens inside heads


# ───────────────────────────── attention ─────────────────────────────

B, S, H, D = 2, 190, 4, 64
NB = B * S * H * D * 2  # of a dense tensor
DENSE, PART = (S * H * D, H * D, D), (S * 4 * H * D, 4 * H * D, D)  # PART: heads of a [b][s][4 h][d] tensor


def _desc(strides, **kw):
    a = AttentionDesc(BF16, B, S, kw.get("sk", S), H, H, D, 0.125, 0)
    for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        setattr(a, n + "_stride", (ctypes.c_longlong * 3)(*strides.get(n, DENSE)))
    a.q_len, a.k_len = kw.get("q_len"), kw.get("k_len")
    return ctypes.byref(a)


def _forward(L, strides=(), q_len=None, k_len=None, ws=X - 4096, **at):
    p = {**{n: X + i * NB for i, n in enumerate(("q", "k", "v", "o", "lse"))}, **at}
    return L.vae_attention(_desc(dict(strides), q_len=q_len, k_len=k_len), p["q"], p["k"], p["v"], p["o"], p["lse"], ws, 1 << 40, None)


def _backward(L, strides=(), q_len=None, k_len=None, **at):
    names = ("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws")
    p = {**{n: X + i * NB for i, n in enumerate(names)}, **at}
    return L.vae_attention_backward(_desc(dict(strides), q_len=q_len, k_len=k_len), *[p[n] for n in names], 1 << 40, None)


def test_attention_refuses_shared_memory(L):
    o, lse = X + 3 * NB, X + 4 * NB
    for kw in (dict(o=X + 16), dict(o=X + NB - 16), dict(o=X + 2 * NB + 128), dict(o=X + 128), dict(lse=o), dict(lse=o + NB - 16),
               dict(lse=X + 32), dict(q_len=o + 64), dict(k_len=lse + 8), dict(q=o - 128, o=o)):
        assert _forward(L, **kw) == -1 and "overlap" in vg.last_error(), kw
    # heads of one projection that do meet
    st = dict(q=PART, o=PART)
    assert _forward(L, st, q=X, o=X + 2 * 3 * D, k=X * 2, v=X * 3, lse=X * 4) == -1
    # rows of o in one another: tokens a head apart, heads and tokens of one stride
    for ostr in ((S * H * D, D, D), (S * H * D, 2 * D, D), (H * D, H * D, D), (S * H * D, H * D, (S - 1) * H * D)):
        assert _forward(L, dict(o=ostr)) == -2 and "row" in vg.last_error(), ostr


def test_attention_workspace_is_checked_where_it_is_used(L):
    """One token over a long cache: the pieces' partial rows."""
    a = AttentionDesc(BF16, 1, 1, 30000, 4, 4, 64, 0.125, 0)
    for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv"):
        setattr(a, n + "_stride", (ctypes.c_longlong * 3)(30000 * 256, 256, 64))
    need = L.vae_attention_workspace_bytes(ctypes.byref(a))
    assert need > 0
    kv, end = X + (1 << 20), X + (1 << 20) + 30000 * 512
    p = (X, kv, end, X + 4096, X + 8192)
    for ws in (X, kv + 4096, kv - need + 16, X + 4096 - need + 16, X + 8192 - need + 16, end + 30000 * 512 - 16):
        assert L.vae_attention(ctypes.byref(a), *p, ws, need, None) == -1 and "overlap" in vg.last_error()


def test_attention_backward_refuses_shared_memory(L):
    names = ("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv")
    at = {n: X + i * NB for i, n in enumerate(names)}
    for w in ("dq", "dk", "dv"):
        for r in names:
            if r != w:
                for off in (16, -16):
                    assert _backward(L, **{w: at[r] + off}) == -1 and "overlap" in vg.last_error(), (w, r)
    for n in names:
        assert _backward(L, ws=at[n] + 16) == -1 and "overlap" in vg.last_error(), n
    assert _backward(L, q_len=at["dk"]) == -1 and _backward(L, k_len=X + 9 * NB + 32) == -1
    for n in ("dq", "dk", "dv"):
        assert _backward(L, {n: (S * H * D, 2 * D, D)}) == -2 and "row" in vg.last_error()


def test_attention_takes_views_that_lie_in_one_another(L, no_gpu):
    part = lambda *n: {x: PART for x in n}  # noqa: E731
    p = lambda i: X + 2 * i * H * D  # noqa: E731
    assert _forward(L) in NO_GPU
    # q, k, v and o beside one another in one tensor
    assert _forward(L, part("q", "k", "v", "o"), q=p(0), k=p(1), v=p(2), o=p(3), lse=X * 4) in NO_GPU
    assert _backward(L, part("dq", "dk", "dv"), dq=X * 2 + 2 * H * D, dk=X * 2 + 4 * H * D, dv=X * 2) in NO_GPU
    # gradients beside what they are of, in one tensor
    assert _backward(L, part("q", "dq"), q=X * 2, dq=X * 2 + 2 * H * D) in NO_GPU
    # heads before tokens, tokens before the batch
    assert _backward(L, dict(do=(S * H * D, D, S * D), dq=(H * D, B * H * D, D))) in NO_GPU
    # inputs may share memory with one another
    assert _forward(L, k=X, v=X) in NO_GPU and _forward(L, q_len=X, k_len=X) in NO_GPU
    # a workspace that is not used is not looked at
    assert _forward(L, ws=X) in NO_GPU
