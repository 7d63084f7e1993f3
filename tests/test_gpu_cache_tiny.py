"""Blocks whose span is among f32's smallest numbers, where a fifteenth or a 127th of it is less than the smallest of them:
the scale is the format's smallest all the same, by the layout's bytes."""
import numpy as np
import pytest

import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import FORMS, Pool, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,dim", FORMS)
def test_scales_of_the_smallest_spans(bits, dim):
    say("tiny", bits, dim)
    p = Pool(bits, 1, dim, 64, [62], seed=dim)
    least = 2.0 ** -149
    for x, sign in ((p.k[0], 1), (p.v[0], -1)):
        x[...] = 0
        for t in range(62):
            x[t, 0, 7::32] = np.float32(sign * least * (t if t < 40 else 2 ** (t - 35)))
        x[::3, 0, 9::32] = np.float32(-least)
    q8.cache_append(p.cache, p.batch(starts=[0, 62], rows=62), _dev(p.k[0]), _dev(p.v[0]))
    got, want = p.cache.data.cpu().numpy(), p.packed([62])
    assert np.array_equal(got, want), len(np.argwhere(got != want))
