"""Queries whose elements lie far apart: a row's largest meets keys of zero and the small ones make the scores.

Beside the bound of cache_reference.py, whose term 2^-21 Z is that of 22 bits of every element: a row is lifted so that its
largest element times scale lies in [2^14, 2^15), and its second words end on binary16's grid of 2^-24.  An element is
off by half of that, 2^-39 of the largest, or by 2^-22 of itself, so a score by |scale| 2^-39 max |q| sum |k_t| more.
"""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import Pool, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 128), (4, 256)])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("power", [12, 20, 28, 36, 60])
def test_elements_far_below_their_rows_largest(bits, dim, new, power):
    say("spread queries", bits, dim, new, power)
    rng = np.random.default_rng(power)
    n, heads = 400, 4
    p = Pool(bits, 1, dim, 64, [n], seed=dim)
    p.k[0][..., :32] = 0
    p.fill()
    q = rng.standard_normal((new, heads, dim)).astype(np.float32)
    q[..., 5] = np.float32(2.0 ** power) * rng.uniform(1, 2, (new, heads)).astype(np.float32)
    q[:, 1] *= np.float32(2.0 ** -power)  # (the same row, lifted the other way)
    out, lse = (t.cpu().numpy().astype(np.float64) for t in q8.attention(p.cache, p.batch(starts=[0, new], rows=new), _dev(q)))
    k, v = p.values(0)
    q = q.astype(np.float64)
    for r in {0, new - 1}:
        at = np.array([n - new + r])
        want, want_lse, bound, lse_bound, _ = ref.attend(q[r:r + 1], k, v, at, 1 / np.sqrt(dim))
        for h in range(heads):
            more = 2.0 ** -39 / np.sqrt(dim) * np.abs(q[r, h]).max() * np.abs(k[:at[0] + 1, 0]).sum(-1).max()
            z = k[:at[0] + 1, 0] @ q[r, h] / np.sqrt(dim)
            w = np.exp(z - z.max())
            size = (w / w.sum()) @ np.abs(v[:at[0] + 1, 0])
            # (weights off by a factor of exp(2 more) at most; a softmax's output never leaves its values' range)
            assert (np.abs(out[r, h] - want[0, h]) <= bound[0, h] + size * np.expm1(min(2 * more, 50))).all(), (r, h)
            assert np.abs(lse[r, h] - want_lse[0, h]) <= lse_bound[0, h] + more, (r, h)
