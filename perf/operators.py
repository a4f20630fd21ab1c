"""Workloads of the operators on latent tokens: layer norm, rotary positions, attention, and their gradients.

Each case is one call as a program makes it around the decoders: tokens of an
image's or a video's latent grid, normalised, rotated by their (time, height,
width) positions, attending to one another within padded batches or from frame
to earlier frames, in both directions. ``run`` computes a case in plain torch
operations, or with ``own`` through the library; ``exact`` gives the operators'
definition in 64 bits.

Attention's rule, as the library documents it: with ql, kl the valid lengths of
a batch entry, query i sits at position i + kl - ql; with ``block`` > 0 it sees
the keys of its own block of ``block`` positions and of the earlier ones, else
every key below kl. A row that sees nothing is 0 (its log-sum-exp -inf); rows
behind ql or kl are left as they were, which is 0 here.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0


# ───────────────────────────── cases ─────────────────────────────

def _ln(name, m, c, x, y, backward):
    return {"name": name, "kind": "layernorm_backward" if backward else "layernorm", "m": m, "c": c, "x": x, "y": y}


def _rope(name, b, frames, height, width, heads, d, t, time_dims, interleaved, inverse):
    """Tokens of b clips of frames x height x width; time_dims of the d head dims turn with
    the frame, the rest half each with the row and the column."""
    return {"name": name, "kind": "rotary", "b": b, "frames": frames, "height": height, "width": width, "heads": heads,
            "d": d, "t": t, "time_dims": time_dims, "interleaved": interleaved, "inverse": inverse}


def _att(name, b, sq, sk, hq, hkv, d, t, block, ragged, backward):
    return {"name": name, "kind": "attention_backward" if backward else "attention", "b": b, "sq": sq, "sk": sk,
            "hq": hq, "hkv": hkv, "d": d, "t": t, "block": block, "ragged": ragged}


def listed():
    return [
        # the tokens of one 16 x 16 latent before a projection: latency counts
        _ln("layernorm 256x512", 256, 512, "f32", "f16", False),
        # a 128 x 128 latent (a 1024 x 1024 image) at the width of the decoder's mid block
        _ln("layernorm 16384x1152", 16384, 1152, "f32", "f16", False),
        # a short, odd training batch in 16 bits
        _ln("layernorm grad 1001x576", 1001, 576, "bf16", "bf16", True),
        # a training batch of four 128 x 128 latents: f32 stream, f16 gradients from the projection
        _ln("layernorm grad 65536x1152", 65536, 1152, "f32", "f16", True),
        # queries and keys of one small image, two axes
        _rope("rotary image 16x16", 1, 1, 16, 16, 16, 64, "bf16", 0, False, False),
        # queries and keys of a video clip, three axes, interleaved pairs
        _rope("rotary video 9x64x64", 1, 9, 64, 64, 18, 128, "f16", 16, True, False),
        # one small image: latency counts
        _att("attention 256 tokens", 1, 256, 256, 8, 8, 64, "f16", 0, False, False),
        # a 128 x 128 latent, every token sees every other
        _att("attention 16384 tokens", 1, 16384, 16384, 9, 9, 128, "f16", 0, False, False),
        # one new token per request over long caches of other lengths, four query heads to a key head
        _att("attention cache 32760", 4, 1, 32760, 16, 4, 128, "bf16", 0, True, False),
        # a small training step in 16 bits
        _att("attention grad 256 tokens", 2, 256, 256, 8, 8, 64, "f16", 0, False, True),
        # a training batch of padded clips, frames of 1024 tokens that see the earlier frames, shared heads
        _att("attention grad frames", 2, 4100, 4100, 16, 4, 96, "bf16", 1024, True, True),
        # training on a 128 x 128 latent
        _att("attention grad 16384 tokens", 1, 16384, 16384, 9, 9, 128, "f16", 0, False, True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["ln", "ln_grad", "rope", "att", "cache", "att_grad"])
    if kind in ("ln", "ln_grad"):
        m, c = _spread(rng, 1, 65536), _spread(rng, 48, 4096)
        c = c if rng.random() < 0.2 else (c + 7) // 8 * 8  # odd widths among them
        m = max(1, min(m, 65536 * 1152 // c // (1 if kind == "ln_grad" else 2)))
        case = _ln("", m, c, rng.choice(list(TYPES)), rng.choice(list(TYPES)), kind == "ln_grad")
    elif kind == "rope":
        d = rng.choice([32, 64, 80, 96, 128])
        h, w = _spread(rng, 4, 96), _spread(rng, 4, 96)
        frames, heads, b = _spread(rng, 1, 17), _spread(rng, 1, 32), rng.randint(1, 3)
        frames = max(1, min(frames, 9 * 64 * 64 * 18 * 128 // (h * w * heads * d * b * 2)))
        time_dims = rng.choice([0, d // 8 // 4 * 4, d // 4])
        time_dims -= (d - time_dims) % 4
        case = _rope("", b, frames, h, w, heads, d, rng.choice(list(TYPES)), max(0, time_dims), rng.random() < 0.5,
                     rng.random() < 0.5)
    else:
        d = rng.choice([40, 64, 72, 96, 128])
        hkv, g, b = rng.choice([1, 2, 3, 4, 8, 9]), rng.choice([1, 1, 2, 3, 4, 8]), rng.randint(1, 4)
        back = kind == "att_grad"
        if kind == "cache":
            sq, sk = rng.choice([1, 1, 1, 2, 5, 16]), _spread(rng, 1, 32768)
        else:
            sq = _spread(rng, 1, 16384)
            sk = sq if rng.random() < 0.6 else _spread(rng, 16, 16384)
        cap = (3.0e11 if back else 1.2e11)  # multiply-adds of one product over all heads, well under the largest case's
        while b * hkv * g * float(sq) * sk * d > cap or b * hkv * g * float(sq) * sk > 1.0e9:
            if b > 1:
                b -= 1
            elif g > 1:
                g -= 1
            elif hkv > 1:
                hkv -= 1
            else:
                sk = max(1, sk // 2)
        block = rng.choice([0, 0, 1, _spread(rng, 2, 1024)])
        case = _att("", b, sq, sk, hkv * g, hkv, d, rng.choice(["f16", "bf16"]), block, rng.random() < 0.5, back)
    del case["name"]
    return case


# ───────────────────────────── inputs ─────────────────────────────

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, t="f32", std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(TYPES[t])

    s = dict(case)
    kind = case["kind"]
    if kind.startswith("layernorm"):
        m, c = case["m"], case["c"]
        # a residual stream: channels of their own mean, rows of their own size
        s["xt"] = (normal(m, c) * (0.5 + torch.rand((m, 1), generator=gen, device="cuda")) + normal(1, c, std=0.5)).to(TYPES[case["x"]])
        s["gamma"], s["beta"] = normal(c, std=0.1, mean=1.0), normal(c, std=0.1)
        if kind == "layernorm_backward":
            s["dy"] = normal(m, c, t=case["y"])
        return s
    if kind == "rotary":
        b, f, h, w = case["b"], case["frames"], case["height"], case["width"]
        s["xt"] = normal(b, f * h * w, case["heads"], case["d"], t=case["t"])
        ax = [torch.arange(n, device="cuda", dtype=torch.float32) for n in (f, h, w)]
        grid = torch.stack(torch.meshgrid(*ax, indexing="ij"), -1).reshape(1, f * h * w, 3)
        # each clip starts at a frame and a place of its own
        start = torch.randint(0, 512, (b, 1, 3), generator=gen, device="cuda").float()
        s["pos"] = (grid + start).contiguous()
        rest = case["d"] - case["time_dims"]
        s["axes"] = (case["time_dims"], rest // 2, rest - rest // 2)
        if own:
            import implicit_gemm_convolution_vae_gb300 as vg
            s["plan"] = vg.RopePlan(s["axes"], theta=THETA, interleaved=case["interleaved"])
        return s
    b, sq, sk, hq, hkv, d, t = (case[k] for k in ("b", "sq", "sk", "hq", "hkv", "d", "t"))
    s["q"], s["k"], s["v"] = normal(b, sq, hq, d, t=t, std=1.5), normal(b, sk, hkv, d, t=t), normal(b, sk, hkv, d, t=t)
    s["q_len"] = s["k_len"] = None
    if case["ragged"]:
        # lengths between half and all of the padded ones, now and then 0 or 1
        def lengths(n):
            v = n - (torch.rand((b,), generator=gen, device="cuda") * (n // 2 + 1)).int()
            few = torch.rand((b,), generator=gen, device="cuda")
            return torch.where(few < 0.05, (few < 0.025).int(), v.clamp(max=n)).int()
        s["k_len"] = lengths(sk)
        s["q_len"] = s["k_len"] if sq == sk else lengths(sq) if sq > 16 else None
    if kind == "attention_backward":
        s["do"] = normal(b, sq, hq, d, t=t)
        o, lse = _attention(s)
        s["o"], s["lse"] = o, lse
    return s


# ───────────────────────────── plain forms ─────────────────────────────

def _layernorm(s):
    x = s["xt"].float()
    x = x - x.mean(1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["gamma"] + s["beta"]
    return y.to(TYPES[s["y"]])


def _layernorm_backward(s):
    x, dy = s["xt"].float(), s["dy"].float()
    x = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    n = x * r
    g = dy * s["gamma"]
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return {"dx": dx.to(TYPES[s["x"]]), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}


def _pairs(s, x):
    """The rotated pairs of x [..., d]: (first, second) of each."""
    return (x[..., 0::2], x[..., 1::2]) if s["interleaved"] else (x[..., :s["d"] // 2], x[..., s["d"] // 2:])


def _rotary(s):
    freq = torch.cat([THETA ** (-torch.arange(0, n, 2, device="cuda", dtype=torch.float64) / max(n, 1)) for n in s["axes"]])
    axis = torch.cat([torch.full((n // 2,), i, device="cuda", dtype=torch.long) for i, n in enumerate(s["axes"])])
    angle = s["pos"].double()[..., axis] * freq  # [b][tokens][pairs]: far positions need the 64 bits
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    if s["inverse"]:
        sin = -sin
    a, b = _pairs(s, s["xt"].float())
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return y.to(TYPES[s["t"]])


def _hidden(s):
    """(pairs that are not seen [b][1][1][sq][sk] or None, valid rows [b][sq], valid keys [b][sk])."""
    b, sq, sk = s["b"], s["sq"], s["sk"]
    full = lambda n: torch.full((b,), n, device="cuda")  # noqa: E731
    ql = full(sq) if s["q_len"] is None else s["q_len"].long()
    kl = full(sk) if s["k_len"] is None else s["k_len"].long()
    i, j = torch.arange(sq, device="cuda"), torch.arange(sk, device="cuda")
    rows, keys = i[None] < ql[:, None], j[None] < kl[:, None]
    if not s["ragged"] and not s["block"]:
        return None, rows, keys
    seen = (rows[:, :, None] & keys[:, None])
    if s["block"]:
        at = i[None] + (kl - ql)[:, None]
        seen = seen & (j // s["block"] <= torch.div(at, s["block"], rounding_mode="floor")[:, :, None])
    return ~seen[:, None, None], rows, keys


def _heads(s, x, h):
    """[b][n][heads][d] -> f32 [b][hkv][heads / hkv][n][d]."""
    b, n, _, d = x.shape
    return x.float().reshape(b, n, s["hkv"], h // s["hkv"], d).permute(0, 2, 3, 1, 4)


def _scores(s):
    hidden, rows, keys = _hidden(s)
    x = _heads(s, s["q"], s["hq"]) @ _heads(s, s["k"], s["hkv"]).transpose(-1, -2) * (1.0 / math.sqrt(s["d"]))
    return (x if hidden is None else x.masked_fill_(hidden, -math.inf)), rows, keys


def _tokens(s, x, t):
    """[b][hkv][g][n][d] -> [b][n][heads][d] in the type t."""
    b, hkv, g, n, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, hkv * g, d).to(TYPES[t])


def _softmax(x):
    """(probabilities, log-sum-exp) of the last axis; a row of -inf gives zeros and -inf."""
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total == 0, 1.0, total)), (top + torch.log(total))[..., 0]


def _attention(s):
    x, rows, keys = _scores(s)
    p, lse = _softmax(x)
    o = _tokens(s, p @ _heads(s, s["v"], s["hkv"]), s["t"])
    return o, lse.reshape(s["b"], s["hq"], s["sq"])


def _attention_backward(s):
    x, rows, keys = _scores(s)
    p, _ = _softmax(x)
    do = _heads(s, s["do"], s["hq"])
    dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
    dp = do @ _heads(s, s["v"], s["hkv"]).transpose(-1, -2)
    dp -= (p * dp).sum(-1, keepdim=True)
    ds = p.mul_(dp).mul_(1.0 / math.sqrt(s["d"]))
    dq = ds @ _heads(s, s["k"], s["hkv"])
    dk = (ds.transpose(-1, -2) @ _heads(s, s["q"], s["hq"])).sum(2, keepdim=True)
    return {"dq": _tokens(s, dq, s["t"]), "dk": _tokens(s, dk, s["t"]), "dv": _tokens(s, dv, s["t"])}


# ───────────────────────────── one pass ─────────────────────────────

def run(state):
    s, kind = state, state["kind"]
    if not own:
        if kind == "layernorm":
            return _layernorm(s)
        if kind == "layernorm_backward":
            return _layernorm_backward(s)
        if kind == "rotary":
            return _rotary(s)
        if kind == "attention":
            o, lse = _attention(s)
            return {"o": o, "lse": lse}
        return _attention_backward(s)
    import implicit_gemm_convolution_vae_gb300 as vg
    if kind == "layernorm":
        return vg.layernorm(s["xt"], s["gamma"], s["beta"], eps=EPS, out_dtype=TYPES[s["y"]])
    if kind == "layernorm_backward":
        dx, dgamma, dbeta = vg.layernorm_backward(s["dy"], s["xt"], s["gamma"], eps=EPS)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if kind == "rotary":
        return vg.rope(s["xt"], s["pos"], s["plan"], inverse=s["inverse"])
    if kind == "attention":
        o, lse = vg.attention(s["q"], s["k"], s["v"], q_len=s["q_len"], k_len=s["k_len"], block=s["block"])
        return {"o": o, "lse": lse}
    dq, dk, dv = vg.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], q_len=s["q_len"],
                                       k_len=s["k_len"], block=s["block"])
    return {"dq": dq, "dk": dk, "dv": dv}


# ───────────────────────────── work ─────────────────────────────

def _size(t):
    return 4 if t == "f32" else 2


def work(case):
    kind = case["kind"]
    if kind == "layernorm":
        m, c = case["m"], case["c"]
        return {"bytes": m * c * (_size(case["x"]) + _size(case["y"])) + 8 * c, "flops": 8 * m * c}
    if kind == "layernorm_backward":
        m, c = case["m"], case["c"]
        return {"bytes": m * c * (2 * _size(case["x"]) + _size(case["y"])) + 12 * c, "flops": 16 * m * c}
    if kind == "rotary":
        n = case["b"] * case["frames"] * case["height"] * case["width"]
        return {"bytes": 2 * n * case["heads"] * case["d"] * _size(case["t"]) + 12 * n, "flops": 3 * n * case["heads"] * case["d"]}
    b, sq, sk, hq, hkv, d, block = (case[k] for k in ("b", "sq", "sk", "hq", "hkv", "d", "block"))
    # a ragged batch holds three quarters of its padded tokens on average; the products of pairs that are seen
    part = 0.75 if case["ragged"] else 1.0
    rows, keys = b * sq * (part if sq > 16 else 1.0), b * sk * part
    if block:
        at = torch.arange(sq, dtype=torch.float64) + (sk - sq)
        seen = ((torch.floor(at / block) + 1) * block).clamp(0, sk).mean().item()
    else:
        seen = float(sk)
    pairs = rows * seen * part * hq
    if kind == "attention":
        return {"bytes": 2 * d * (2 * rows * hq + 2 * keys * hkv) + 4 * rows * hq, "flops": 4 * d * pairs}
    return {"bytes": 2 * d * (4 * rows * hq + 4 * keys * hkv) + 4 * rows * hq, "flops": 10 * d * pairs}


# ───────────────────────────── the definitions in 64 bits ─────────────────────────────

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("layernorm"):
        x = s["xt"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        hat = (x - mean) / torch.sqrt(var + EPS)
        if kind == "layernorm":
            return hat * s["gamma"].double() + s["beta"].double()
        dy = s["dy"].double()
        # the gradient through hat, projected off the row's constant and off hat itself
        up = dy * s["gamma"].double()
        along = (up * hat).sum(1, keepdim=True) / case["c"]
        dx = (up - up.sum(1, keepdim=True) / case["c"] - hat * along) / torch.sqrt(var + EPS)
        return {"dx": dx, "dgamma": torch.einsum("mc,mc->c", dy, hat), "dbeta": torch.einsum("mc->c", dy)}
    if kind == "rotary":
        # one complex number per pair, turned by its angle
        turn = torch.cat([s["pos"][..., i:i + 1].double() / THETA ** (torch.arange(n // 2, device="cuda").double() * 2 / max(n, 1))
                          for i, n in enumerate(s["axes"])], -1)
        z = s["xt"].double()
        d, two = case["d"], case["interleaved"]
        z = z.unflatten(-1, (d // 2, 2)) if two else z.unflatten(-1, (2, d // 2)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn)[:, :, None]
        z = torch.view_as_real(z)
        return (z if two else z.transpose(-1, -2)).flatten(-2)
    b, sq, sk, hq, hkv, d, block = (case[k] for k in ("b", "sq", "sk", "hq", "hkv", "d", "block"))
    if b * hq * float(sq) * sk * d * (5 if kind == "attention_backward" else 2) > 3e12:
        return None
    zeros = lambda n, h: torch.zeros((b, n, h, d), dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = zeros(sq, hq), torch.full((b, hq, sq), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = zeros(sq, hq), zeros(sk, hkv), zeros(sk, hkv)
    for e in range(b):
        nq = sq if s["q_len"] is None else int(s["q_len"][e])
        nk = sk if s["k_len"] is None else int(s["k_len"][e])
        for h in range(hq):
            kh = h // (hq // hkv)
            q, k, v = s["q"][e, :nq, h].double(), s["k"][e, :nk, kh].double(), s["v"][e, :nk, kh].double()
            x = torch.mm(q, k.t()) / math.sqrt(d)
            if block:
                last = torch.div(torch.arange(nq, device="cuda") + (nk - nq), block, rounding_mode="floor")
                x[torch.div(torch.arange(nk, device="cuda"), block, rounding_mode="floor")[None] > last[:, None]] = -math.inf
            z = torch.logsumexp(x, 1) if nk else torch.full((nq,), -math.inf, dtype=torch.float64, device="cuda")
            lse[e, h, :nq] = z
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
            out = torch.mm(p, v)
            o[e, :nq, h] = out
            if kind == "attention_backward":
                g = s["do"][e, :nq, h].double()
                dv[e, :nk, kh] += torch.mm(p.t(), g)
                w = p * (torch.mm(g, v.t()) - (g * out).sum(1, keepdim=True)) / math.sqrt(d)
                dq[e, :nq, h] = torch.mm(w, k)
                dk[e, :nk, kh] += torch.mm(w.t(), q)
    return {"o": o, "lse": lse} if kind == "attention" else {"dq": dq, "dk": dk, "dv": dv}
