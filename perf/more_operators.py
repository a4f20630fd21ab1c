"""Workloads of two more operators on latent tokens: the norm of query and key heads with the rotary positions
in one pass, and the gated feed-forward block, with their gradients.

Each case is one call as a program makes it between the projections and
attention, or behind attention, in a block of a model that makes latents:
forward with few tokens or whole grids of them, backward in training. ``run``
computes a case in plain torch operations, or with ``own`` through the library;
``exact`` gives the operators' definition in 64 bits.

The rules, as the library documents them. Norm and rotation of a head x of d
channels: n = x / sqrt(mean(x^2) + eps), y = the pairs of n * gamma turned by
the token's angles. Gated feed-forward: gate = x Wg^T, up = x Wu^T,
hidden = act(gate) * up, y = hidden Wd^T; the gradient is taken at gate, up and
hidden as the forward pass saved them, in the tensors' type.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")
EPS = 1e-6
THETA = 10000.0


# ───────────────────────────── cases ─────────────────────────────

def _qk(name, b, frames, height, width, hq, hk, d, t, time_dims, space_dims, interleaved, joint, backward):
    """Tokens of b clips of frames x height x width; time_dims of the d head dims turn with the frame, space_dims half
    each with the row and the column, the rest not. joint: q and k are parts of one projection's rows."""
    return {"name": name, "kind": "qk_backward" if backward else "qk", "b": b, "frames": frames, "height": height,
            "width": width, "hq": hq, "hk": hk, "d": d, "t": t, "time_dims": time_dims, "space_dims": space_dims,
            "interleaved": interleaved, "joint": joint}


def _ffn(name, m, c, f, t, activation, backward):
    return {"name": name, "kind": "ffn_backward" if backward else "ffn", "m": m, "c": c, "f": f, "t": t,
            "activation": activation}


def listed():
    return [
        # one new token for each of eight requests, on its way into their caches: latency counts
        _qk("qk norm 8 single tokens", 8, 1, 1, 1, 16, 4, 128, "bf16", 0, 128, False, True, False),
        # queries and keys of one small image
        _qk("qk norm image 16x16", 1, 1, 16, 16, 8, 8, 64, "f16", 0, 64, False, True, False),
        # queries and keys of a video clip, three axes, interleaved pairs
        _qk("qk norm video 9x64x64", 1, 9, 64, 64, 18, 18, 128, "f16", 16, 112, True, True, False),
        # a short, odd training batch in 32 bits, heads of which a part turns
        _qk("qk norm grad 2x7x11x13", 2, 7, 11, 13, 6, 2, 72, "f32", 8, 48, True, False, True),
        # training on a video clip, shared key heads
        _qk("qk norm grad video 9x64x64", 1, 9, 64, 64, 18, 6, 128, "bf16", 16, 112, False, True, True),
        # one new token: the weights are read once
        _ffn("ffn 1 token", 1, 1152, 4608, "bf16", "silu", False),
        # the tokens of one 16 x 16 latent
        _ffn("ffn 256 tokens", 256, 512, 2048, "f16", "silu", False),
        # odd sizes, which end inside tiles
        _ffn("ffn 1001 tokens 584x1560", 1001, 584, 1560, "bf16", "gelu", False),
        # a 128 x 128 latent (a 1024 x 1024 image) at the width of the decoder's mid block
        _ffn("ffn 16384 tokens", 16384, 1152, 4608, "bf16", "silu", False),
        # a small training step
        _ffn("ffn grad 256 tokens", 256, 512, 2048, "f16", "silu", True),
        # a ragged training batch
        _ffn("ffn grad 4100 tokens 576x2304", 4100, 576, 2304, "bf16", "gelu_tanh", True),
        # training on a 128 x 128 latent
        _ffn("ffn grad 16384 tokens", 16384, 1152, 4608, "bf16", "silu", True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["qk", "qk_single", "qk_grad", "ffn", "ffn_few", "ffn_grad"])
    if kind.startswith("qk"):
        d = rng.choice([32, 40, 64, 72, 80, 96, 128])
        hq = _spread(rng, 1, 32)
        hk = rng.choice([hq, hq, max(1, hq // 2), max(1, hq // 4), 1])
        if kind == "qk_single":
            b, frames, h, w = _spread(rng, 1, 256), 1, 1, 1
        else:
            b, frames, h, w = rng.randint(1, 3), _spread(rng, 1, 17), _spread(rng, 4, 96), _spread(rng, 4, 96)
            most = 9 * 64 * 64 * 24 * 128  # elements of q and k together
            frames = max(1, min(frames, most // (b * h * w * (hq + hk) * d)))
        turned = d if rng.random() < 0.7 else d // 2 // 4 * 4
        time_dims = rng.choice([0, turned // 8 // 4 * 4, turned // 4 // 4 * 4])
        time_dims += (turned - time_dims) % 4
        return _without_name(_qk("", b, frames, h, w, hq, hk, d, rng.choice(list(TYPES)), time_dims, turned - time_dims,
                                 rng.random() < 0.5, rng.random() < 0.5, kind == "qk_grad"))
    back = kind == "ffn_grad"
    m = _spread(rng, 1, 48) if kind == "ffn_few" else _spread(rng, 1, 32768)
    c = (_spread(rng, 64, 2304) + 7) // 8 * 8
    f = (int(c * rng.uniform(1.0, 4.0)) + 7) // 8 * 8
    m = max(1, min(m, 16384 * 1152 * 4608 // (c * f)))
    return _without_name(_ffn("", m, c, f, rng.choice(["f16", "bf16"]), rng.choice(ACTIVATIONS), back))


def _without_name(case):
    del case["name"]
    return case


# ───────────────────────────── inputs ─────────────────────────────

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, t="f32", std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(TYPES[t])

    s = dict(case)
    if case["kind"].startswith("qk"):
        b, f, h, w, hq, hk, d, t = (case[k] for k in ("b", "frames", "height", "width", "hq", "hk", "d", "t"))
        n = f * h * w
        # heads of their own size, as a projection gives them
        if case["joint"]:
            rows = normal(b, n, hq + 2 * hk, d, t=t, std=1.5)  # (the values' heads stand behind the keys')
            s["q"], s["k"] = rows[:, :, :hq], rows[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(b, n, hq, d, t=t, std=1.5), normal(b, n, hk, d, t=t, std=0.7)
        s["gamma_q"], s["gamma_k"] = normal(d, std=0.2, mean=1.0), normal(d, std=0.2, mean=1.0)
        ax = [torch.arange(i, device="cuda", dtype=torch.float32) for i in (f, h, w)]
        grid = torch.stack(torch.meshgrid(*ax, indexing="ij"), -1).reshape(1, n, 3)
        # each clip starts at a frame and a place of its own
        s["pos"] = (grid + torch.randint(0, 512, (b, 1, 3), generator=gen, device="cuda").float()).contiguous()
        half = case["space_dims"] // 4 * 2
        s["axes"] = (case["time_dims"], half, case["space_dims"] - half)
        if case["kind"] == "qk_backward":
            s["dq"], s["dk"] = normal(b, n, hq, d, t=t), normal(b, n, hk, d, t=t)
        if own:
            import implicit_gemm_convolution_vae_gb300 as vg
            s["plan"] = vg.RopePlan(s["axes"], theta=THETA, interleaved=case["interleaved"])
        return s
    m, c, f, t = (case[k] for k in ("m", "c", "f", "t"))
    s["x"] = normal(m, c, t=t)  # rows behind a norm
    s["w_gate"], s["w_up"] = normal(f, c, t=t, std=1.5 / math.sqrt(c)), normal(f, c, t=t, std=1.0 / math.sqrt(c))
    s["w_down"] = normal(c, f, t=t, std=1.0 / math.sqrt(f))
    if case["kind"] == "ffn_backward":
        s["dy"] = normal(m, c, t=t)
        # what the forward pass saved
        gate, up = s["x"].float() @ s["w_gate"].float().T, s["x"].float() @ s["w_up"].float().T
        s["hidden"] = (_act(gate, case["activation"])[0] * up).to(TYPES[t])
        s["gate"], s["up"] = gate.to(TYPES[t]), up.to(TYPES[t])
    return s


# ───────────────────────────── plain forms ─────────────────────────────

def _angles(s):
    """(cos, sin) of every token's pairs, [b][tokens][1][pairs] f32."""
    freq = torch.cat([THETA ** (-torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / max(n, 1)) for n in s["axes"]])
    axis = torch.cat([torch.full((n // 2,), i, device="cuda", dtype=torch.long) for i, n in enumerate(s["axes"])])
    angle = s["pos"].double()[..., axis] * freq  # far positions need the 64 bits
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _turn(s, x, cos, sin):
    """The pairs of x [b][tokens][heads][d] turned; channels behind the turned ones as they are."""
    turned = 2 * cos.shape[-1]
    z = x[..., :turned]
    a, b = (z[..., 0::2], z[..., 1::2]) if s["interleaved"] else (z[..., :turned // 2], z[..., turned // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    z = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((z, x[..., turned:]), -1)


def _normed(x):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _qk_heads(s, x, gamma, cos, sin):
    return _turn(s, _normed(x)[0] * gamma, cos, sin).to(TYPES[s["t"]])


def _qk_heads_backward(s, dy, x, gamma, cos, sin):
    n, r = _normed(x)
    u = _turn(s, dy.float(), cos, -sin)
    v = u * gamma
    return (r * (v - n * (v * n).mean(-1, keepdim=True))).to(TYPES[s["t"]]), (u * n).sum((0, 1, 2))


def _act(x, kind):
    """(the activation, its derivative) of an f32 tensor."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    if kind == "gelu":
        p = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    k, a = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(k * (x + a * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3.0 * a * x * x)


def _ffn_forward(s):
    x = s["x"].float()
    hidden = _act(x @ s["w_gate"].float().T, s["activation"])[0] * (x @ s["w_up"].float().T)
    return (hidden @ s["w_down"].float().T).to(TYPES[s["t"]])


def _ffn_backward(s):
    t = TYPES[s["t"]]
    dy, x = s["dy"].float(), s["x"].float()
    dh = dy @ s["w_down"].float()
    value, slope = _act(s["gate"].float(), s["activation"])
    dgate, dup = dh * s["up"].float() * slope, dh * value
    return {"dx": (dgate @ s["w_gate"].float() + dup @ s["w_up"].float()).to(t), "dw_gate": (dgate.T @ x).to(t),
            "dw_up": (dup.T @ x).to(t), "dw_down": (dy.T @ s["hidden"].float()).to(t)}


# ───────────────────────────── one pass ─────────────────────────────

def run(state):
    s, kind = state, state["kind"]
    if not own:
        if kind == "ffn":
            return _ffn_forward(s)
        if kind == "ffn_backward":
            return _ffn_backward(s)
        cos, sin = _angles(s)
        if kind == "qk":
            return {"q": _qk_heads(s, s["q"], s["gamma_q"], cos, sin), "k": _qk_heads(s, s["k"], s["gamma_k"], cos, sin)}
        dq, dgq = _qk_heads_backward(s, s["dq"], s["q"], s["gamma_q"], cos, sin)
        dk, dgk = _qk_heads_backward(s, s["dk"], s["k"], s["gamma_k"], cos, sin)
        return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}
    import implicit_gemm_convolution_vae_gb300 as vg
    if kind == "ffn":
        return vg.gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], activation=s["activation"])
    if kind == "ffn_backward":
        dx, dw_gate, dw_up, dw_down = vg.gated_ffn_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"],
                                                            (s["gate"], s["up"], s["hidden"]), activation=s["activation"])
        return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up, "dw_down": dw_down}
    if kind == "qk":
        q, k = vg.qk_norm_rope(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["pos"], s["plan"], eps=EPS)
        return {"q": q, "k": k}
    dq, dk, dgq, dgk = vg.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["pos"],
                                                s["plan"], eps=EPS)
    return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}


# ───────────────────────────── work ─────────────────────────────

def work(case):
    back = case["kind"].endswith("backward")
    if case["kind"].startswith("qk"):
        tokens = case["b"] * case["frames"] * case["height"] * case["width"]
        n = tokens * (case["hq"] + case["hk"]) * case["d"]
        size = 4 if case["t"] == "f32" else 2
        return {"bytes": n * size * (3 if back else 2) + 12 * tokens + 8 * case["d"] * (2 if back else 1),
                "flops": n * (16 if back else 8)}
    m, c, f = case["m"], case["c"], case["f"]
    if back:
        return {"bytes": 2 * (3 * m * c + 3 * m * f + 6 * c * f), "flops": 12 * m * c * f}
    return {"bytes": 2 * (2 * m * c + 3 * c * f), "flops": 6 * m * c * f}


# ───────────────────────────── the definitions in 64 bits ─────────────────────────────

def _exact_act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x), torch.sigmoid(x) + x * torch.sigmoid(x) * torch.sigmoid(-x)
    if kind == "gelu":
        cdf = 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x * x / 2.0) / math.sqrt(2.0 * math.pi)
    # 0.5 (1 + tanh(z)) is the logistic function of 2 z
    z2 = 2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
    p = torch.sigmoid(z2)
    return x * p, p + x * p * torch.sigmoid(-z2) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * x ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("ffn"):
        x, wg, wu, wd = (s[k].double() for k in ("x", "w_gate", "w_up", "w_down"))
        if kind == "ffn":
            value, _ = _exact_act(torch.einsum("mc,fc->mf", x, wg), case["activation"])
            return torch.einsum("mf,cf->mc", value.mul_(torch.einsum("mc,fc->mf", x, wu)), wd)
        dy = s["dy"].double()
        dh = torch.einsum("mc,cf->mf", dy, wd)
        value, slope = _exact_act(s["gate"].double(), case["activation"])
        dup = value.mul_(dh)
        dgate = slope.mul_(dh).mul_(s["up"].double())
        dx = torch.einsum("mf,fc->mc", dgate, wg) + torch.einsum("mf,fc->mc", dup, wu)
        return {"dx": dx, "dw_gate": torch.einsum("mf,mc->fc", dgate, x), "dw_up": torch.einsum("mf,mc->fc", dup, x),
                "dw_down": torch.einsum("mc,mf->cf", dy, s["hidden"].double())}
    # one complex number per pair, turned by its angle
    turns = torch.cat([s["pos"][..., i:i + 1].double() / THETA ** (torch.arange(n // 2, device="cuda").double() * 2 / max(n, 1))
                       for i, n in enumerate(s["axes"])], -1)
    phase = torch.polar(torch.ones_like(turns), turns)[:, :, None]
    pairs, two = turns.shape[-1], case["interleaved"]

    def turned(x, by):
        z = x[..., :2 * pairs]
        z = z.unflatten(-1, (pairs, 2)) if two else z.unflatten(-1, (2, pairs)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        return torch.cat(((z if two else z.transpose(-1, -2)).flatten(-2), x[..., 2 * pairs:]), -1)

    out = {}
    for i in "qk":
        x, gamma = s[i].double(), s["gamma_" + i].double()
        size = torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS)
        if kind == "qk":
            out[i] = turned(x / size * gamma, phase)
            continue
        up = turned(s["d" + i].double(), phase.conj())
        out["dgamma_" + i] = torch.einsum("bshd,bshd->d", up, x / size)
        # through the norm: what is left of up * gamma once its part along x is taken off
        along = torch.einsum("bshd,bshd->bsh", up * gamma, x)[..., None] / (case["d"] * size * size)
        out["d" + i] = (up * gamma - along * x) / size
    return out
