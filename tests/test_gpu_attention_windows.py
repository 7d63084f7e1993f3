"""Windows as wide as the call takes, beside rows before the first token: they hide nothing.

Checked as in test_gpu_attention.py, whose reference and bounds these tests use; the call without a
window gives the same bits, since it sees the same tokens.
"""
import numpy as np
import pytest
import torch

import q8_projection_amd as q8
from helpers import say
from test_gpu_attention import check
from test_gpu_cache import Pool, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 128), (4, 256)])
@pytest.mark.parametrize("group,new", [(1, 7), (1, 16), (2, 8), (4, 40), (1, 300)])
@pytest.mark.parametrize("window", [2 ** 30 - 1, 2 ** 30, 2 ** 31 - 300, 2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1])
def test_windows_that_hide_nothing(bits, dim, group, new, window):
    """Up to all of a sequence's rows lie before its first token; 16 rows or fewer and more are other kernels."""
    say("wide window", bits, dim, group, new, window)
    lens = [max(1, new - 5), 2, 0, new + 90, new]
    p = Pool(bits, 2, dim, 32, lens, seed=group + new).fill()
    q = normal(np.random.default_rng(4), 5 * new, 2 * group, dim)
    got = check(p, lens, [new] * 5, 2 * group, window=window, q=q, sample=3)
    batch = p.batch(starts=np.arange(6) * new, rows=5 * new, max_rows=new)
    want = q8.attention(p.cache, batch, torch.from_numpy(q).cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
