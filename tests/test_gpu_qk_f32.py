"""The heads' norm in f32 at every way that a row's 32-byte units lie over lanes: one lane a
row, odd numbers of units, units without a neighbour, parts that do not turn. Bounds and
checks are those of test_gpu_qk.py."""
import pytest

import test_gpu_qk as qk

pytestmark = pytest.mark.gpu

# b, s, hq, hk, d, axes, type, interleaved, int positions, per batch, gammas
CASES = [(1, 70, 3, 2, d, axes, "f32", inter, False, True, True)
         for d, axes in ((8, (8,)), (8, None), (16, (8, 8)), (16, (4,)), (24, (16, 8)), (32, (32,)), (40, (16,)), (48, (16, 32)), (56, (4, 20, 20)),
                         (72, (24, 24, 24)), (88, (80,)), (104, (32,)), (128, (64, 64)), (136, (128,)), (200, (96, 96)), (248, (16,)), (256, (128, 128)))
         for inter in (True, False)]
CASES += [(2, 3000, 5, 3, 128, (64, 64), "f32", False, True, False, True), (1, 9001, 2, 1, 40, (20, 20), "f32", False, False, True, True)]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    qk.test_qk_norm_rope(case)


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    qk.test_qk_norm_rope_backward(case)
