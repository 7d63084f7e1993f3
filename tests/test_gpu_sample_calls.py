"""Calls of the sampler whose parameters meet in ways that its other tests do not."""
import numpy as np
import pytest

from helpers import say
from test_gpu_sample import check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n", [(1, 151936), (3, 524287), (40, 30011)])
def test_the_largest_logit_of_a_row_with_filters_set(rows, n):
    """Temperatures at or below zero, or NaN, on rows long enough for several workgroups,
    with min-p (and other filters) on: one workgroup answers."""
    say("greedy", rows, n)
    l = logits_of(rows, n, 5 * n + rows)
    l[:, n // 3] = l[:, n - 2] = l.max(axis=1) + 1  # two of them: the lower index
    for t in (0.0, -0.0, -1.0, float("nan")):
        for kw in (dict(min_p=0.1), dict(min_p=1e-9), dict(min_p=2.0), dict(min_p=0.1, top_k=3000), dict(min_p=0.1, top_p=0.5)):
            idx, prob = check(l, temperature=t, what=(t, kw), **kw)
            assert (idx == n // 3).all() and (prob == np.float32(1)).all()


@pytest.mark.filterwarnings("ignore:invalid value encountered in cast")
def test_signaling_nan_is_no_candidate_either():
    l = logits_of(4, 5003, 43)
    bits = l.view(np.uint32)
    bits[0, 1::2] = 0x7f800001
    bits[1, ::3] = 0xff800001
    bits[2, :] = 0x7fbfffff
    bits[3, ::64] = 0x7fa00000
    for kw in (dict(), dict(top_k=20), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0), dict(top_k=4000)):
        check(l, what=kw, **kw)
