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
