"""What the binding of the heads' norm and of the gated feed-forward block refuses by
itself (CPU only): with its own error, before anything is packed for the library."""
import pytest

import implicit_gemm_convolution_vae_gb300 as vg


@pytest.mark.parametrize("saved", [(), (1, 2), (1, 2, 3, 4), "abc"])
def test_saved_values_that_are_no_three(saved):
    import torch
    x, w, d = torch.zeros(2, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    saved = tuple(w for _ in saved) if isinstance(saved, tuple) else saved
    with pytest.raises(vg.VaeError, match="saved"):
        vg.gated_ffn_backward(x, x, w, w, d, saved)


@pytest.mark.parametrize("eps", [1e39, -1e39])
def test_an_eps_that_f32_does_not_hold(eps):
    import torch
    vg._torch()
    q = torch.zeros(1, 2, 3, 8)
    with pytest.raises(vg.VaeError, match="eps"):
        vg._qk_desc(q, q, None, None, None, None, eps, q, q)


def test_positions_of_more_batch_entries_than_the_desc_holds():
    import torch
    vg._torch()
    q = torch.zeros(1, 1, 3, 8)
    plan = vg.RopePlan((8,))
    pos = torch.empty(1 << 31, 1, 1, dtype=torch.int32, device="meta")
    with pytest.raises(vg.VaeError, match="positions"):
        vg._qk_desc(q, q, None, None, pos, plan, 1e-6, q, q)
