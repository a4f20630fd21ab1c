"""Sizes that the C ABI's 31 bits do not hold are refused by the binding (CPU
only): ctypes would pass their low bits on, and the call would take a part of
the tensor for the whole."""
import pytest

import implicit_gemm_convolution_vae_gb300 as vg
from implicit_gemm_convolution_vae_gb300.build import build

FAR = (1 << 32) + 4  # its low 32 bits: 4


@pytest.fixture(scope="module", autouse=True)
def library():
    build()
    vg._torch()


def _meta(*shape, t="float16"):
    import torch
    return torch.empty(shape, dtype=getattr(torch, t), device="meta")


@pytest.mark.parametrize("shape", [(FAR, 1), (1, FAR)])
def test_layernorm_refuses_sizes_over_31_bits(shape):
    x = _meta(*shape)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg._layernorm(x, None, None, 1e-6, None, x, None)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg._layernorm_backward(x, x, None, 1e-6, False, x, None, None, None, None)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg.layernorm_backward_workspace_bytes(*shape)


@pytest.mark.parametrize("shape", [(FAR, 1, 1, 8), (1, FAR, 1, 8), (1, 1, FAR, 8), (1, 1, 1, FAR)])
def test_rope_and_attention_refuse_sizes_over_31_bits(shape):
    x = _meta(*shape)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg._rope(x, _meta(shape[1], 1, t="float32"), vg.RopePlan((8,)), False, x, None)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg._attention(x, x, x, None, None, None, 0, x, None, None, None)
    with pytest.raises(vg.VaeError, match="below 2.31"):
        vg._attention_backward(x, x, x, x, x, None, None, None, None, 0, x, x, x, None, None)


@pytest.mark.parametrize("which", range(7))
def test_attention_workspaces_refuse_sizes_over_31_bits(which):
    sizes = [1, 4, 4, 2, 2, 64, 0]
    sizes[which] = FAR
    for f in (vg.attention_workspace_bytes, vg.attention_backward_workspace_bytes):
        with pytest.raises(vg.VaeError, match="below 2.31"):
            f(*sizes)


def test_rope_plan_refuses_axes_over_31_bits():
    for axes in ((FAR,), (8, -FAR)):
        with pytest.raises(vg.VaeError, match="below 2.31"):
            vg.RopePlan(axes)
