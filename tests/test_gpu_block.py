"""The operators of a token block together, as a model and its training call them:
norms, projections, the norm of query and key heads with rotary positions, attention over
frames, the gated feed-forward block; forward, back, and from several threads."""
import threading

import numpy as np
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from gpu_common import torch_mod
from oracle import tokens as ot
from vae_inputs import rng_for

pytestmark = pytest.mark.gpu


def _draw(name, shape, t, std=1.0, mean=0.0):
    torch = torch_mod()
    a = rng_for(30, "block." + name).standard_normal(shape) * std + mean
    x = torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    return x, x.double().cpu().numpy()


def _np(x):
    return x.double().cpu().numpy()


def test_whole_block_forward_and_backward():
    """norm -> joint projection -> heads' norm and rotation -> attention over frames -> output projection with the residual ->
    norm -> gated feed-forward with the residual, and the gradient of every input and weight of the two parts; against
    float64. About twenty roundings of half an f16 step (2^-11) lie between input and output in either direction, and
    scores of a few units move p by 2^-8 at most: 2^-7 of the norm, 2^-6 for the gradients that pass both parts."""
    torch = torch_mod()
    b, f, s, hq, hk, d, hid = 2, 3, 50, 4, 2, 32, 136
    c, n, block = hq * d, f * s, s
    m, h3 = b * n, hq + 2 * hk
    f16, f32 = torch.float16, torch.float32
    x, x64 = _draw("x", (m, c), f32)
    g1, g1r = _draw("g1", (c,), f32, 0.2, 1.0)
    g2, g2r = _draw("g2", (c,), f32, 0.2, 1.0)
    gq, gqr = _draw("gq", (d,), f32, 0.2, 1.0)
    gk, gkr = _draw("gk", (d,), f32, 0.2, 1.0)
    wp, wpr = _draw("wp", (h3 * d, c), f16, 1.0 / np.sqrt(c))
    wo, wor = _draw("wo", (c, c), f16, 1.0 / np.sqrt(c))
    wg, wgr = _draw("wg", (hid, c), f16, 1.0 / np.sqrt(c))
    wu, wur = _draw("wu", (hid, c), f16, 1.0 / np.sqrt(c))
    wd, wdr = _draw("wd", (c, hid), f16, 1.0 / np.sqrt(hid))
    dout, doutr = _draw("dout", (m, c), f16)
    grid = torch.stack(torch.meshgrid(torch.arange(f), torch.arange(5), torch.arange(10), indexing="ij"), -1).reshape(n, 3)
    pos, axes = grid.to(torch.int32).cuda(), (8, 12, 12)
    plan = vg.RopePlan(axes)
    # forward
    y = vg.layernorm(x, g1, out_dtype=f16)
    rows = vg.conv1x1(y, wp, out_f16=True).view(b, n, h3, d)
    q0, k0, v = rows[:, :, :hq], rows[:, :, hq:hq + hk], rows[:, :, hq + hk:]
    q, k = vg.qk_norm_rope(q0, k0, gq, gk, pos, plan)
    o, lse = vg.attention(q, k, v, block=block)
    x2 = vg.conv1x1(o.view(m, c), wo, residual=x)
    z = vg.layernorm(x2, g2, out_dtype=f16)
    out, saved = vg.gated_ffn(z, wg, wu, wd, residual=x2, save=True)
    # backward: the gradient of the stream in f32, that of each part's output in f16
    dz, dwg, dwu, dwd = vg.gated_ffn_backward(dout, z, wg, wu, wd, saved, grad_dtype=f32)
    dx2, dg2, _ = vg.layernorm_backward(dz, x2, g2)
    dx2 = dx2 + dout.float()
    do = vg.conv1x1(dx2.half(), wo.t().contiguous(), out_f16=True).view(b, n, hq, d)
    dq, dk, dv = vg.attention_backward(do, q, k, v, o, lse, block=block)
    drows = torch.empty_like(rows)
    drows[:, :, hq + hk:] = dv
    _, _, dgq, dgk = vg.qk_norm_rope_backward(dq, dk, q0, k0, gq, gk, pos, plan, dq=drows[:, :, :hq], dk=drows[:, :, hq:hq + hk])
    dy = vg.conv1x1(drows.view(m, h3 * d), wp.t().contiguous())
    dx, dg1, _ = vg.layernorm_backward(dy, x, g1)
    dx = dx + dx2
    vg.sync_status()
    # float64
    p = grid.numpy()
    yr = ot.layernorm(x64, g1r)
    rr = (yr @ wpr.T).reshape(b, n, h3, d)
    q0r, k0r, vr = rr[:, :, :hq], rr[:, :, hq:hq + hk], rr[:, :, hq + hk:]
    qr, kr = ot.qk_norm_rope(q0r, gqr, p, axes), ot.qk_norm_rope(k0r, gkr, p, axes)
    orr, _ = ot.attention(qr, kr, vr, block=block)
    x2r = orr.reshape(m, c) @ wor.T + x64
    zr = ot.layernorm(x2r, g2r)
    fr, gater, upr, hidr = ot.gated_ffn(zr, wgr, wur, wdr)
    outr = fr + x2r
    dzr, dwgr, dwur, dwdr, _, _ = ot.gated_ffn_backward(doutr, zr, wgr, wur, wdr, gater, upr, hidr)
    dx2r, dg2r, _ = ot.layernorm_backward(dzr, x2r, g2r)
    dx2r = dx2r + doutr
    dqr, dkr, dvr = ot.attention_backward((dx2r @ wor).reshape(b, n, hq, d), qr, kr, vr, block=block)
    dq0r, dgqr = ot.qk_norm_rope_backward(dqr, q0r, gqr, p, axes)
    dk0r, dgkr = ot.qk_norm_rope_backward(dkr, k0r, gkr, p, axes)
    dyr = np.concatenate((dq0r, dk0r, dvr), 2).reshape(m, h3 * d) @ wpr
    dxr, dg1r, _ = ot.layernorm_backward(dyr, x64, g1r)
    dxr = dxr + dx2r
    off = lambda a, r: np.linalg.norm(_np(a) - r) / np.linalg.norm(r)  # noqa: E731
    for got, ref in ((out, outr), (dwg, dwgr), (dwu, dwur), (dwd, dwdr), (dg2, dg2r)):
        assert off(got, ref) <= 2.0 ** -7
    for got, ref in ((dx, dxr), (dg1, dg1r), (dgq, dgqr), (dgk, dgkr)):
        assert off(got, ref) <= 2.0 ** -6


def test_one_token_after_another_into_a_cache():
    """Serving: each step's keys go straight to their place in a cache, and the block's rows are those of the whole sequence
    at once. The two differ in how attention tiles its rows and the products their sums, a few roundings in bf16: 2^-6."""
    torch = torch_mod()
    b, n, hq, hk, d, hid = 3, 9, 4, 2, 64, 264
    c, bf = hq * d, torch.bfloat16
    rows, _ = _draw("srv.rows", (b, n, hq + 2 * hk, d), bf)
    gq, gk = _draw("srv.gq", (d,), torch.float32, 0.2, 1.0)[0], _draw("srv.gk", (d,), torch.float32, 0.2, 1.0)[0]
    wg, wu, wd = (_draw("srv." + i, sh, bf, 0.08)[0] for i, sh in (("g", (hid, c)), ("u", (hid, c)), ("d", (c, hid))))
    plan = vg.RopePlan((d,))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    q, k = vg.qk_norm_rope(rows[:, :, :hq], rows[:, :, hq:hq + hk], gq, gk, pos, plan)
    o, _ = vg.attention(q, k, rows[:, :, hq + hk:], block=1)
    whole = vg.gated_ffn(o.view(b * n, c), wg, wu, wd).view(b, n, c)
    kc = torch.full((b, 16, hk, d), float("nan"), dtype=bf, device="cuda")
    vc = kc.clone()
    for i in range(n):
        vc[:, i] = rows[:, i, hq + hk:]
        qi, _ = vg.qk_norm_rope(rows[:, i:i + 1, :hq], rows[:, i:i + 1, hq:hq + hk], gq, gk, pos[i:i + 1], plan, k_out=kc[:, i:i + 1])
        lens = torch.full((b,), i + 1, dtype=torch.int32, device="cuda")
        oi, _ = vg.attention(qi, kc, vc, k_len=lens)
        yi = vg.gated_ffn(oi.view(b, c), wg, wu, wd)
        assert (yi.float() - whole[:, i].float()).norm() <= 2.0 ** -6 * whole[:, i].float().norm()
    assert torch.equal(kc[:, :n], k) and kc[:, n:].isnan().all()


def test_calls_of_other_sizes_from_several_threads():
    """Plans and set-up are shared between calls; results are those of one thread."""
    torch = torch_mod()
    sizes = [(1, 64, 136), (40, 264, 520), (300, 136, 264), (700, 200, 72), (2500, 72, 520)]
    work = []
    for m, c, f in sizes:
        x, wg, wu, wd = (torch.randn(s, device="cuda").mul_(0.2).bfloat16() for s in ((m, c), (f, c), (f, c), (c, f)))
        q, k = torch.randn(1, m, 3, 64, device="cuda").half(), torch.randn(1, m, 1, 64, device="cuda").half()
        y, saved = vg.gated_ffn(x, wg, wu, wd, save=True)
        work.append((x, wg, wu, wd, q, k, saved, (y, *vg.gated_ffn_backward(y, x, wg, wu, wd, saved), *vg.qk_norm_rope(q, k))))
    torch.cuda.synchronize()
    wrong = []

    def turn(first):
        stream = torch.cuda.Stream()
        for i in range(30):
            x, wg, wu, wd, q, k, saved, ref = work[(first + i) % len(work)]
            got = (vg.gated_ffn(x, wg, wu, wd, stream=stream),
                   *vg.gated_ffn_backward(ref[0], x, wg, wu, wd, saved, stream=stream), *vg.qk_norm_rope(q, k, stream=stream))
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, ref)):
                wrong.append((first, i))

    threads = [threading.Thread(target=turn, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    vg.sync_status()
