"""Attention of many rows: row tiles that are shared, taken whole, or spread over rounds of sequences.

Checked as in test_gpu_attention.py, whose reference and bounds these tests use.
"""
import numpy as np
import pytest
import torch

import q8_projection_amd as q8
from helpers import say
from test_gpu_attention import check
from test_gpu_cache import FORMS, Pool, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("group,new", [(1, 33), (4, 40), (6, 3), (8, 100)])
def test_row_tiles_that_many_workgroups_share(bits, dim, group, new):
    """A few row tiles after a long cached part: every one has many parts, of two sequences of unequal lengths."""
    say("shared", bits, dim, group, new)
    lens = [6000, 1111]
    p = Pool(bits, 2, dim, 64, lens, seed=dim + new).fill()
    check(p, lens, [new, new], 2 * group, sample=6)
    check(p, lens, [new, new - 1], 2 * group, window=1500, sample=6)


@pytest.mark.parametrize("bits,dim", FORMS)
def test_prompts_of_whole_and_of_shared_row_tiles(bits, dim):
    """From a row tile for a few workgroups to several for each."""
    say("sizes", bits, dim)
    for heads, lens in ((4, [500]), (8, [1200]), (16, [900, 1100, 40])):
        p = Pool(bits, 4, dim, 64, lens, seed=len(lens)).fill()
        check(p, lens, lens, heads, sample=5)
        check(p, lens, [n - 1 for n in lens], heads, window=200, sample=5)


@pytest.mark.parametrize("dim", [64, 256])
def test_rows_of_more_sequences_than_a_wave_has_lanes(dim):
    say("rounds", dim)
    rng = np.random.default_rng(dim)
    lens = [int(n) for n in rng.integers(0, 120, 150)]
    lens[100] = 2500
    news = [min(int(m), n) for m, n in zip(rng.integers(0, 60, 150), lens)]
    news[3] = news[70] = 0
    p = Pool(4, 1, dim, 32, lens, seed=5).fill()
    check(p, lens, news, 4, sample=2)
    check(p, [n if 64 <= s < 128 else 0 for s, n in enumerate(lens)], [n if 64 <= s < 128 else 0 for s, n in enumerate(news)], 4, sample=2)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_token_of_more_heads_than_a_row_tile_has_rows(dim):
    say("heads", dim)
    p = Pool(4, 1, dim, 64, [700, 90], seed=dim).fill()
    check(p, [700, 90], [1, 1], 300, starts=False, sample=1)
    check(p, [700, 90], [3, 2], 300, window=100, sample=3)


@pytest.mark.parametrize("starts,lens", [([0, 40, 80], [2 ** 31 - 1, -5]), ([-7, 40, 80], [60, 70]), ([0, 2 ** 31 - 1, 80], [60, 70]),
                                         ([80, 40, 0], [60, 70]), ([-2 ** 31, 2 ** 31 - 1, -1], [60, 70]), ([0, 40, 10 ** 6], [-2 ** 31, 70])])
@pytest.mark.parametrize("dim", [128, 256])
def test_starts_and_lengths_that_make_no_sense_reach_no_other_memory(starts, lens, dim):
    say("starts", starts, lens, dim)
    p = Pool(4, 2, dim, 32, [60, 70], seed=1).fill()
    around = torch.full((84, 8, dim), 7.0, device="cuda")
    lse = torch.full((84, 8), 7.0, device="cuda")
    batch = p.batch(lens=lens, starts=starts, rows=80, max_rows=40)
    q8.attention(p.cache, batch, torch.randn((80, 8, dim), device="cuda"), out=around[2:82], lse=lse[2:82])
    # (the rows themselves may see tokens that were never written)
    assert (around[:2] == 7).all() and (around[82:] == 7).all() and (lse[:2] == 7).all() and (lse[82:] == 7).all()


def test_one_workspace_serves_every_kernel_and_size():
    say("workspace")
    pools = [Pool(bits, 2, dim, 64, [1500, 200], seed=dim).fill() for bits, dim in ((4, 64), (8, 128), (4, 256))]
    work = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    first = {}
    for turn in range(3):
        for i, p in enumerate(pools):
            for new in (1, 30, 200):
                q = normal(np.random.default_rng(new), 2 * new, 8, p.dim)
                got = check(p, [1500, 200], [new, new], 8, q=q, workspace=work, sample=1)
                if turn == 0:
                    first[i, new] = got
                assert all(torch.equal(a, b) for a, b in zip(got, first[i, new])), (turn, i, new)


def test_captured_calls_with_workspaces_of_their_own():
    """Two graphs, one of single tokens and one of chunks, replayed by turns and at once."""
    say("graphs")
    p = Pool(4, 2, 128, 64, [2000, 300], seed=3).fill()
    calls, kept = [], []
    for new in (1, 60):
        batch = p.batch(starts=[0, new, 2 * new], rows=2 * new, max_rows=new)
        q = torch.randn((2 * new, 8, 128), device="cuda")
        work = q8.attention_workspace(p.cache, batch, 8)
        want = q8.attention(p.cache, batch, q, workspace=work)
        out = [torch.empty_like(t) for t in want]
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q8.attention(p.cache, batch, q, out=out[0], lse=out[1], workspace=work)
        calls.append((graph, stream, out, want))
        kept.append((batch, q, work))  # a graph does not
    for _ in range(4):
        for graph, stream, out, want in calls:
            out[0].fill_(3.0), out[1].fill_(3.0)
        torch.cuda.synchronize()
        for graph, stream, out, want in calls:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, out, want in calls:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
