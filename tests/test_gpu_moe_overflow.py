"""An expert layer in the f32 mode whose inputs are finite and whose h overflows f32.

h is rounded to f32, so one that is too large is infinite, and every later value of
that token is the formula's: an infinity of the down weight's sign.  Nothing is
rounded in the expected values: they are 0, infinities, or one product that is exact.
The down weights are quants without a zero (0 times infinity would be NaN in the
formula too) and scale 1.  Both kinds of kernels, and each way of splitting the steps.
"""
import numpy as np
import pytest
import torch

import q8_projection_amd as q8
from helpers import say

pytestmark = pytest.mark.gpu

K = 64


def blocks(quants):
    """Q8_0 blocks of scale 1 for int8 quants [experts][n][k]."""
    e, n, k = quants.shape
    out = np.zeros((e, n, k // 32, 34), np.uint8)
    out[..., :2] = np.array([1.0], np.float16).view(np.uint8)
    out[..., 2:] = quants.reshape(e, n, k // 32, 32).view(np.uint8)
    return torch.from_numpy(out.reshape(e, n, k // 32 * 34)).cuda()


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 40])  # up to 3 on vector instructions, then on the matrix cores
@pytest.mark.parametrize("ff,at", [(64, 5), (2048, 7), (2048, 1300), (2048, 2047), (2112, 1056), (2112, 2111), (8256, 4127),
                                   (14336, 9000)])
def test_an_h_that_overflows_is_an_infinity_of_y(rows, ff, at):
    say("overflow", rows, ff, at)
    rng = np.random.default_rng(ff + at)
    gate = np.zeros((1, ff, K), np.int8)
    gate[0, at, 0] = 1                                  # g = u = x[0] in h's element `at`, 0 in the others
    down = (rng.integers(1, 100, (1, K, ff)) * rng.choice([-1, 1], (1, K, ff))).astype(np.int8)
    layer = q8.MoeLayer("f32", blocks(gate), blocks(gate), blocks(down), K, ff, 1)
    x = np.zeros((rows, K), np.float32)
    x[:, 0] = 1024.0                                    # h = 2^20: sigmoid(1024) is 1 in f64
    x[:, 1] = rng.normal(size=rows)
    x[rows // 2, 0] = 1e20                              # h = 1e40
    ids = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    y = q8.moe_experts(layer, torch.from_numpy(x).cuda(), ids, torch.ones((rows, 1), device="cuda"))
    torch.cuda.synchronize()
    h = np.full((rows, 1), 2.0 ** 20)
    h[rows // 2] = np.inf
    assert np.array_equal(y.cpu().numpy(), (h * down[0, :, at].astype(np.float64)).astype(np.float32))
