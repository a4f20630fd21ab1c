"""The norm of query and key heads at its largest number of tokens, 2^31 - 256: the rows
at both ends and around the middle are those of a short call, bit for bit, whichever form
takes them (a scalar a lane, vectors with their positions). The other rows are zeros."""
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from gpu_common import torch_mod
from vae_inputs import rng_for

pytestmark = pytest.mark.gpu

TOKENS = (1 << 31) - 256
PLACES = [slice(a, a + 40) for a in (0, (1 << 30) - 21, TOKENS // 2 + 7, TOKENS - 40)]


def _draw(name, shape, t):
    torch = torch_mod()
    return torch.from_numpy(rng_for(9, "qk.far." + name).standard_normal(shape)).to(t).cuda()


def _spread(short):
    """The rows of `short` [1][160][1][d] at their places among zeros."""
    torch = torch_mod()
    x = torch.zeros(1, TOKENS, 1, short.shape[3], dtype=short.dtype, device="cuda")
    for i, at in enumerate(PLACES):
        x[:, at] = short[:, 40 * i:40 * i + 40]
    return x


def _gather(x, dim=1):
    return torch_mod().cat([x.narrow(dim, at.start, 40) for at in PLACES], dim)


@pytest.mark.parametrize("d,t", [(1, "float16"), (8, "bfloat16")])
def test_qk_norm_rope_at_its_largest_number_of_tokens(d, t):
    torch = torch_mod()
    t = getattr(torch, t)
    q, k, g = _draw("q", (1, 160, 1, d), t), _draw("k", (1, 160, 1, d), t), _draw("g", (d,), torch.float32)
    pos = plan = far = None
    if d > 1:
        plan = vg.RopePlan((d,), interleaved=False)
        pos = torch.arange(160, dtype=torch.int32, device="cuda")[:, None] * 3
        far = torch.zeros(TOKENS, 1, dtype=torch.int32, device="cuda")
        for i, at in enumerate(PLACES):
            far[at] = pos[40 * i:40 * i + 40]
    ref = vg.qk_norm_rope(q, k, g, g, pos, plan)
    a, c = _spread(q), _spread(k)
    vg.qk_norm_rope(a, c, g, g, far, plan, q_out=a, k_out=c)
    assert torch.equal(_gather(a), ref[0]) and torch.equal(_gather(c), ref[1])
    # zeros on both sides of the places stay zeros (the two around the middle are 60 tokens apart)
    for at in PLACES:
        for r in (slice(max(0, at.start - 32), at.start), slice(at.stop, min(TOKENS, at.stop + 32))):
            assert (a[:, r] == 0).all() and (c[:, r] == 0).all()
    # the gradient in place of dy, every token's head the same row
    one, two = _draw("one", (1, 1, 1, d), t), _draw("two", (1, 1, 1, d), t)
    ref = vg.qk_norm_rope_backward(q, k, one.expand(1, 160, 1, d), two.expand(1, 160, 1, d), g, g, pos, plan)
    for x, short in ((a, q), (c, k)):
        x.zero_()
        for i, at in enumerate(PLACES):
            x[:, at] = short[:, 40 * i:40 * i + 40]
    got = vg.qk_norm_rope_backward(a, c, one.expand(1, TOKENS, 1, d), two.expand(1, TOKENS, 1, d), g, g, far, plan, dq=a, dk=c)
    assert torch.equal(_gather(a), ref[0]) and torch.equal(_gather(c), ref[1])
    # dgamma's sums are joined in another order: 160 terms of at most |dy| sqrt(d), 2^-24 of each for every addition
    for x, y, dy in ((got[2], ref[2], q), (got[3], ref[3], k)):
        assert ((x - y).abs() <= 2 * 160 * 2.0 ** -24 * d ** 0.5 * dy.float().abs().sum()).all()
    vg.sync_status()
