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
