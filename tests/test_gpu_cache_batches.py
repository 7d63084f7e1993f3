"""A batch of sequences used with more than one cache."""
import pytest
import torch

import q8_projection_amd as q8

pytestmark = pytest.mark.gpu


def test_a_batch_serves_caches_of_other_page_sizes():
    """What a batch knows of its workspace's size is of the cache that it is asked for."""
    table = torch.zeros((1, 1 << 19), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    long, short = (q8.KVCache(4, 1, 64, page, 1) for page in (4096, 32))
    batch = q8.CacheBatch(short, table, lens)
    assert q8.attention_workspace_bytes(long, batch, 1) == 0  # more than 2^30 tokens
    assert q8.attention_workspace_bytes(short, batch, 1) > 0
    short.data.zero_()
    out, _ = q8.attention(short, batch, torch.ones((1, 1, 64), device="cuda"))
    assert (out == 0).all()
