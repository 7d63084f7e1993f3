"""Sequences of one call that have the same pages: chunks of one prompt, one token each, meet anywhere in a
tile, in the same bytes too.  The pool's every byte against the layout's formulas, as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import FORMS, Pool, _dev

pytestmark = pytest.mark.gpu


def append_in_chunks(p, cuts, shuffled):
    """One call: each sequence of the pool cut into chunks at cuts[s], a chunk being a sequence of the call."""
    table, lens, k, v = [], [], [], []
    for s, at in enumerate(cuts):
        ends = [0, *at, int(p.lens[s])]
        for a, b in zip(ends[:-1], ends[1:]):
            table.append(p.table[s])
            lens.append(b)
            k.append(p.k[s][a:b])
            v.append(p.v[s][a:b])
    order = p.rng.permutation(len(lens)) if shuffled else np.arange(len(lens))
    news = [len(k[i]) for i in order]
    batch = q8.CacheBatch(p.cache, _dev(np.stack([table[i] for i in order])), _dev(np.array([lens[i] for i in order], np.int32)),
                          _dev(np.concatenate([[0], np.cumsum(news)]).astype(np.int32)), sum(news), max(news))
    q8.cache_append(p.cache, batch, _dev(np.concatenate([k[i] for i in order])), _dev(np.concatenate([v[i] for i in order])))


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("shuffled", [False, True])
def test_chunks_that_meet_within_a_tile(bits, dim, shuffled):
    say("chunks", bits, dim, shuffled)
    p = Pool(bits, 2, dim, 64, [41, 70, 9, 33, 66], entries=3)
    cuts = [[37], [1, 2, 3, 33, 35, 42, 67], [4], [31, 32], [5, 13, 29, 30, 31, 34, 40, 61]]
    append_in_chunks(p, cuts, shuffled)
    assert np.array_equal(p.cache.data.cpu().numpy(), p.packed(p.lens))


@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_of_one_prompt_as_sequences_of_one_token(bits):
    """Every token's codes are written by a wave of its own."""
    say("tokens as sequences", bits)
    p = Pool(bits, 2, 64, 128, [129, 300, 31], entries=3)
    append_in_chunks(p, [list(range(1, n)) for n in p.lens], True)
    assert np.array_equal(p.cache.data.cpu().numpy(), p.packed(p.lens))


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 128)])
def test_many_chunks_of_many_prompts(bits, dim):
    """Chunks of three tokens, thousands at once, read back; then the same tokens written over other codes."""
    say("many chunks", bits, dim)
    lens = [200] * 40
    p = Pool(bits, 4, dim, 64, lens, seed=dim)
    starts = np.arange(41) * 200
    for turn in range(3):
        append_in_chunks(p, [list(range(3 - turn, 200, 3)) for _ in lens], True)
        k, v = q8.cache_read(p.cache, p.batch(starts=starts, rows=8000, max_rows=200))
        for got, x in ((k, p.k), (v, p.v)):
            assert np.array_equal(got.cpu().numpy().astype(np.float64), ref.values(bits, np.concatenate(x))), turn
        p.k, p.v = p.v, p.k


@pytest.mark.parametrize("bits", [4, 8])
def test_chunks_that_meet_within_a_tile_replayed(bits):
    """A captured call over pages that other tokens are in by now."""
    say("chunks, replayed", bits)
    p = Pool(bits, 2, 128, 64, [50, 50], seed=6)
    table, lens = _dev(p.table[[0, 0, 1, 1]]), _dev(np.array([13, 50, 29, 50], np.int32))
    batch = q8.CacheBatch(p.cache, table, lens, _dev(np.array([0, 13, 50, 79, 100], np.int32)), 100, 37)
    k, v = torch.empty((100, 2, 128), device="cuda"), torch.empty((100, 2, 128), device="cuda")
    k.normal_(), v.normal_()
    q8.cache_append(p.cache, batch, k, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.cache_append(p.cache, batch, k, v)
    for turn in range(4):
        for s in (0, 1):
            p.k[s], p.v[s] = p.k[s][::-1].copy(), (p.v[s] * (turn + 1)).astype(np.float32)
        k.copy_(_dev(np.concatenate(p.k)))
        v.copy_(_dev(np.concatenate(p.v)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(p.cache.data.cpu().numpy(), p.packed([50, 50])), turn
