"""Calls whose launches are sized by max_rows far above what the sequences have."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import normal

pytestmark = pytest.mark.gpu


def test_more_work_than_a_launch_has_workgroups():
    """Rows of 20000 sequences of which any might have had all: the workgroups go round."""
    say("many")
    n = 20000
    cache = q8.KVCache(4, 1, 64, 32, n)
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0).contiguous()[:, None]
    at = torch.arange(n, dtype=torch.int32, device="cuda") % 32
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    batch = q8.CacheBatch(cache, table, at + 1, starts, rows=n)
    rng = np.random.default_rng(7)
    k, v = normal(rng, n, 1, 64), normal(rng, n, 1, 64)
    q8.cache_append(cache, batch, torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    got = q8.cache_read(cache, batch)
    assert np.array_equal(got[0].cpu().numpy(), ref.values(4, k)) and np.array_equal(got[1].cpu().numpy(), ref.values(4, v))
    # one token a sequence is seen in a window of one: its value
    out, _ = q8.attention(cache, batch, torch.randn((n, 1, 64), device="cuda"), window=1)
    want = torch.from_numpy(ref.values(4, v).astype(np.float32)).cuda()
    # (a weight exp(0) in two words is exact up to f32's roundings: the product, the sum, the quotient)
    assert ((out - want).abs() <= 4 * torch.finfo(torch.float32).eps * want.abs()).all()
