"""Attention over the quantized cache against the formulas in 64 bits.

The reference takes the values that the cache stands for (binary16 numbers) and the f32
queries; the bounds are cache_reference.py's, for each output and for the errors' 2-norm.
"""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import FORMS, Pool, _dev, normal

pytestmark = pytest.mark.gpu


def check(p, lens, news, heads, window=0, scale=None, q=None, starts=True, max_rows=None, have=None, workspace=None, seed=0,
          sample=None):
    """One call over the pool's sequences (news[s] rows each) against the reference.  have[s]: which tokens there are."""
    rng = np.random.default_rng(seed)
    rows, dim = int(sum(news)), p.dim
    q = normal(rng, rows, heads, dim) if q is None else q
    begin = np.concatenate([[0], np.cumsum(news)])
    batch = p.batch(lens=lens, starts=begin, rows=rows, max_rows=max_rows or max(news)) if starts else p.batch(lens=lens)
    out, lse = q8.attention(p.cache, batch, _dev(q), scale=scale, window=window, workspace=workspace)
    torch.cuda.synchronize()
    got, got_lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for s, (n, new) in enumerate(zip(lens, news)):
        if not new:
            continue
        at = n - new + np.arange(new)
        k, v = p.values(s)
        take = np.arange(new) if sample is None else np.unique(np.r_[0, new - 1, rng.integers(0, new, sample)])
        r = begin[s] + take
        want, want_lse, bound, lse_bound, usual = ref.attend(q[r].astype(np.float64), k[:n], v[:n], at[take],
                                                      1 / np.sqrt(dim) if scale is None else np.float64(np.float32(scale)),
                                                      window, None if have is None else have[s][:n])
        err = np.abs(got[r] - want)
        assert (err <= bound).all(), (s, n, new, float((err - bound).max()), float(err.max()))
        assert np.linalg.norm(err) <= np.linalg.norm(usual), (s, n, new, np.linalg.norm(err) / np.linalg.norm(want))
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(got_lse[r])) and (got[r][none] == 0).all()
        assert (np.abs(got_lse[r][~none] - want_lse[~none]) <= lse_bound[~none]).all(), (s, n, new)
    return out, lse


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("group", [1, 4, 7])
def test_single_tokens(bits, dim, group):
    """A decode step of sequences of every small length, empty slots among them."""
    say("tokens", bits, dim, group)
    lens = [0, 1, 2, 31, 32, 33, 63, 64, 65, 0, 127, 200, 257, 0]
    p = Pool(bits, 2, dim, 64, lens, seed=group).fill()
    check(p, lens, [1] * len(lens), 2 * group, starts=False)
    check(p, lens, [1] * len(lens), 2 * group, starts=False, window=40)


@pytest.mark.parametrize("bits,dim,group,page", [(4, 128, 4, 64), (4, 128, 16, 32), (4, 64, 1, 32), (4, 256, 2, 128), (8, 128, 8, 64),
                                                 (8, 64, 3, 32), (8, 256, 1, 64), (4, 128, 17, 64), (4, 128, 32, 64), (8, 64, 31, 64)])
@pytest.mark.parametrize("lens", [[1500], [700, 3, 1100]])
def test_single_tokens_of_long_sequences(bits, dim, group, page, lens):
    say("long", bits, dim, group, page, lens)
    p = Pool(bits, 2, dim, page, lens, entries=50, seed=dim + group).fill()
    check(p, lens, [1] * len(lens), 2 * group, starts=False)
    check(p, lens, [1] * len(lens), 2 * group, starts=False, window=333)


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("group,news", [(4, [3, 1, 4, 2]), (1, [16, 9, 1, 5]), (5, [6, 6, 6, 6]), (8, [1, 0, 4, 1])])
def test_a_few_rows(bits, dim, group, news):
    say("few", bits, dim, group, news)
    lens = [3, 200, 67, 640]
    p = Pool(bits, 2, dim, 32, lens, seed=group).fill()
    for window in (0, 50, 1):
        check(p, lens, news, 2 * group, window=window)


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("group,window", [(1, 0), (4, 0), (6, 33), (1, 100)])
def test_prompts(bits, dim, group, window):
    """Whole prompts of several lengths, one after a cached part, one of a single row, an empty one."""
    say("prompts", bits, dim, group, window)
    lens, news = [130, 1, 33, 0, 257, 64], [130, 1, 33, 0, 120, 64]
    p = Pool(bits, 2, dim, 64, lens, seed=group + window).fill()
    check(p, lens, news, 2 * group, window=window, sample=40)


def test_a_chunk_of_a_prompt_after_a_long_cached_part():
    say("chunk")
    p = Pool(4, 2, 128, 64, [4100, 2000], seed=8).fill()
    check(p, [4100, 2000], [70, 200], 8, sample=12)
    check(p, [4100, 2000], [70, 200], 8, window=1000, sample=12)
    check(p, [4100, 2000], [9, 33], 8, sample=12)


@pytest.mark.parametrize("bits,dim", [(4, 128), (8, 64), (4, 256)])
@pytest.mark.parametrize("news", [[1, 1, 1], [40, 33, 50]])
def test_rows_that_see_nothing_and_pages_that_are_none(bits, dim, news):
    """More rows than tokens, pages outside the pool, tokens past the table's end."""
    say("nothing", bits, dim, news)
    page = 32
    p = Pool(bits, 2, dim, page, [20, 100, 160], entries=4, seed=4)
    p.fill()
    bad = p.table.copy()
    bad[1, 1], bad[1, 3] = p.cache.pages, -1
    good, p.table = p.table, bad
    have = [np.ones(20, bool), np.ones(100, bool), np.arange(160) < 128]
    have[1][32:64] = have[1][96:] = False
    check(p, [20, 100, 160], news, 8, have=have)
    check(p, [20, 100, 160], news, 8, have=have, window=37)
    # every page of a sequence gone: nothing is seen
    p.table = good.copy()
    p.table[:] = 2 ** 31 - 1
    batch = p.batch(lens=[20, 100, 160], starts=np.concatenate([[0], np.cumsum(news)]), rows=sum(news), max_rows=max(news))
    out, lse = q8.attention(p.cache, batch, torch.ones((sum(news), 8, dim), device="cuda"))
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("rows_each", [1, 20])
def test_rows_of_no_sequence_are_left(rows_each):
    p = Pool(4, 2, 128, 32, [50, 60], seed=2).fill()
    rows = 2 * rows_each + 3
    q = torch.randn((rows, 8, 128), device="cuda")
    out, lse = torch.full((rows, 8, 128), 7.0, device="cuda"), torch.full((rows, 8), 7.0, device="cuda")
    batch = p.batch(starts=[0, rows_each, 2 * rows_each], rows=rows, max_rows=rows_each)
    q8.attention(p.cache, batch, q, out=out, lse=lse)
    assert (out[2 * rows_each:] == 7).all() and (lse[2 * rows_each:] == 7).all() and (out[:2 * rows_each] != 7).all()
    # a sequence of more rows than max_rows: the rest are left, too
    out.fill_(7.0)
    batch = p.batch(starts=[0, rows_each + 2, 2 * rows_each + 3], rows=rows, max_rows=rows_each)
    q8.attention(p.cache, batch, q, out=out, lse=lse)
    assert (out[rows_each:rows_each + 2] == 7).all() and (out[rows_each + 2] != 7).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("garbage", [0x00, 0x7f, 0xff, 0x80])
@pytest.mark.parametrize("new", [1, 40])
def test_what_lies_behind_the_tokens_does_not_matter(bits, garbage, new):
    """Codes and words of tokens that are not there: NaN and infinity patterns among the scales."""
    p = Pool(bits, 2, 128, 64, [45, 97], seed=6)
    p.cache.data.fill_(garbage)
    p.fill()
    check(p, [45, 97], [new, new], 8)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new", [1, 40])
def test_large_and_small_values(bits, new):
    """Scores that spread over thousands, keys and values at binary16's ends, queries far below and above them."""
    say("magnitudes", bits, new)
    rng = np.random.default_rng(3)
    for kf, vf, qf, scale in ((1, 1, 30, 3.0), (6e4, 6e4, 1e-9, 0.1), (1e-6, 1e-5, 1e4, 100.0), (1, 1e-6, 1e-30, 1e30), (100, 1, 1e20, 1e-22),
                              (1, 1, 1, 0.0), (1, 1, 1, -0.4)):
        p = Pool(bits, 1, 128, 32, [100], seed=5)
        p.k = [(rng.uniform(-1, 1, (100, 1, 128)) * kf).astype(np.float32)]
        p.v = [(rng.uniform(-1, 1, (100, 1, 128)) * vf).astype(np.float32)]
        p.fill()
        q = (rng.standard_normal((new, 4, 128)) * qf).astype(np.float32)
        q[:, 1] = 0
        q[:, 2] *= 1e-5
        check(p, [100], [new], 4, scale=scale, q=q)


def test_many_sequences():
    """More sequences than a wave has lanes, lengths from none to many."""
    say("many")
    rng = np.random.default_rng(12)
    lens = [int(n) for n in rng.integers(0, 90, 200)]
    lens[150] = 1300
    p = Pool(4, 1, 64, 32, lens, seed=13).fill()
    check(p, lens, [1] * 200, 4, starts=False)
    news = [int(n) for n in rng.integers(0, 4, 200)]
    check(p, lens, news, 4)


@pytest.mark.parametrize("new", [1, 3, 33])
def test_one_workspace_serves_call_after_call(new):
    """The counters are zero again after every call, of other shapes too; the same bits every time."""
    say("workspace", new)
    p = Pool(4, 2, 128, 64, [2500, 40, 900], seed=7).fill()
    lens, news = [2500, 40, 900], [new] * 3
    batch = p.batch(starts=np.arange(4) * new, rows=3 * new, max_rows=new)
    work = torch.zeros(max(q8.attention_workspace_bytes(p.cache, batch, 32), q8.attention_workspace_bytes(p.cache, batch, 8)),
                       dtype=torch.uint8, device="cuda")
    first = check(p, lens, news, 8, workspace=work)
    for _ in range(3):
        check(p, lens, news, 32, workspace=work, sample=1)
        check(p, [100, 40, 900], news, 8, workspace=work, window=64, sample=1)
        again = check(p, lens, news, 8, workspace=work, sample=1)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_queries_in_a_wider_buffer_and_without_lse():
    p = Pool(4, 2, 128, 64, [300, 77], seed=9).fill()
    fused = torch.randn((2, 8 * 128 + 2 * 2 * 128 + 64), device="cuda")
    batch = p.batch()
    q = fused[:, 64:64 + 8 * 128].unflatten(1, (8, 128))
    a, _ = q8.attention(p.cache, batch, q)
    b, _ = q8.attention(p.cache, batch, q.contiguous())
    assert torch.equal(a, b)
    out = torch.empty_like(a)
    work = q8.attention_workspace(p.cache, batch, 8)
    status = q8.lib().q8_attention(p.cache._ref, batch._ref, q.data_ptr(), q.stride(0), 8, 128 ** -0.5, 0, out.data_ptr(), None,
                                   work.data_ptr(), work.numel(), torch.cuda.current_stream().cuda_stream)
    assert status == 0 and torch.equal(out, a)


@pytest.mark.parametrize("new", [1, 2, 50])
def test_other_streams_and_two_at_once(new):
    """Two calls at once on streams and workspaces of their own."""
    p = Pool(4, 2, 128, 64, [3000, 500], seed=10).fill()
    batch = p.batch(starts=[0, new, 2 * new], rows=2 * new, max_rows=new)
    q = [torch.randn((2 * new, 8, 128), device="cuda") for _ in range(2)]
    want = [q8.attention(p.cache, batch, x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [q8.attention(p.cache, batch, x, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_append_and_attention_on_a_stream_of_their_own():
    p = Pool(4, 2, 128, 64, [300], seed=10)
    stream = torch.cuda.Stream()
    k, v = _dev(p.k[0]), _dev(p.v[0])
    torch.cuda.synchronize()
    q8.cache_append(p.cache, p.batch(starts=[0, 300], rows=300), k, v, stream=stream)
    got = q8.cache_read(p.cache, p.batch(starts=[0, 300], rows=300), stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), ref.values(4, p.k[0]))
