"""Calls as large as they come: more pieces and row tiles than a launch has workgroups, pools and rows past 32 bits of
bytes, arrays with guards around them."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import Pool, _dev, normal

pytestmark = pytest.mark.gpu

N, KV, DIM, ENTRIES = 20000, 4, 64, 96


class Many:
    """20000 sequences of up to 32 tokens and a few of 3000, zeros but for the last token: what it adds is known."""

    def __init__(self, rng):
        self.lens = np.arange(N) % 32 + 1
        self.long = [0, 7000, 13337, N - 1]
        self.lens[self.long] = 3000
        table = np.full((N, ENTRIES), -1, np.int32)
        table[:, 0] = np.arange(N)[::-1]
        first = N
        for s in self.long:
            table[s, 1:94] = np.arange(first, first + 93)
            first += 93
        self.cache = q8.KVCache(4, KV, DIM, 32, first)
        self.cache.data.zero_()
        self.table, self.lens_dev = _dev(table), _dev(self.lens.astype(np.int32))
        self.k, self.v = normal(rng, N, KV, DIM), normal(rng, N, KV, DIM)
        q8.cache_append(self.cache, self.batch(None), _dev(self.k), _dev(self.v))

    def batch(self, max_rows):
        starts = None if max_rows is None else torch.arange(N + 1, dtype=torch.int32, device="cuda")
        return q8.CacheBatch(self.cache, self.table, self.lens_dev, starts, N, max_rows)


@pytest.mark.parametrize("max_rows", [None, 32, 33, N])
def test_more_pieces_than_a_launch_has_workgroups(max_rows):
    """80000 sequences and kv heads: workgroups take piece after piece (up to 32 rows), or row tile after row tile, which
    are whole here whatever they cost.  Some sequences are divided and joined among them."""
    say("go round", max_rows)
    rng = np.random.default_rng(3)
    many = Many(rng)
    q = normal(rng, N, KV, DIM)
    out, lse = q8.attention(many.cache, many.batch(max_rows), _dev(q))
    # a token's score z among lens - 1 scores of 0 of tokens whose values are 0
    k, v = ref.values(4, many.k), ref.values(4, many.v)
    z = (k * q.astype(np.float64)).sum(-1) / np.sqrt(DIM)
    others = many.lens[:, None] - 1.0
    want_lse = np.logaddexp(z, np.log(np.maximum(others, 1e-300)))
    p = np.exp(z - want_lse)
    most = (np.abs(k) * np.abs(q)).sum(-1) / np.sqrt(DIM)
    # cache_reference.py's bound; one token alone adds to a sum of values, all of them to the sum of weights
    ez = most * (2.0 ** -21 + (DIM + 8) * 2.0 ** -24) + 8 * 2.0 ** -24 * (1 + np.abs(z))
    chain = (many.lens[:, None] / 8 + 64) * 2.0 ** -24
    err = np.abs(lse.cpu().numpy() - want_lse)
    assert (err <= ez + chain + 2.0 ** -23 * np.abs(want_lse)).all(), np.argwhere(err > ez + chain + 2.0 ** -23 * np.abs(want_lse))[:5]
    top = np.where(others > 0, np.maximum(z, 0.0), z)
    bound = p[..., None] * np.abs(v) * (2 * ez + 2.0 ** -20 + chain)[..., None] + \
        (2.0 ** -36 * np.exp(top - want_lse))[..., None] * np.abs(v)
    off = np.abs(out.cpu().numpy() - p[..., None] * v) > bound
    assert not off.any(), np.argwhere(off)[:5]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new", [1, 90])
def test_pools_past_32_bits_of_bytes(bits, new):
    """The pages at both ends of a pool of some 9 GB, alternating."""
    say("large pool", bits, new)
    small = Pool(bits, 2, 128, 32, [200, 170], seed=bits)
    page = small.cache.data.shape[1]
    pages = (9 << 30) // page
    assert pages * page > 2 * (1 << 32)
    cache = q8.KVCache(bits, 2, 128, 32, pages)
    table = small.table.copy()
    table[:, ::2] += pages - small.cache.pages  # the last pages (the small pool's are at most its number)
    calls = []
    for c, t in ((small.cache, small.table), (cache, table)):
        fill = q8.CacheBatch(c, _dev(t), _dev(small.lens), _dev(np.array([0, 200, 370], np.int32)), 370, 200)
        q8.cache_append(c, fill, _dev(np.concatenate(small.k)), _dev(np.concatenate(small.v)))
        batch = q8.CacheBatch(c, _dev(t), _dev(small.lens), _dev(np.array([0, new, 2 * new], np.int32)), 2 * new, new)
        q = _dev(normal(np.random.default_rng(5), 2 * new, 4, 128))
        calls.append((*q8.cache_read(c, fill), *q8.attention(c, batch, q)))
    assert all(torch.equal(a, b) for a, b in zip(*calls))
    assert np.array_equal(calls[1][0].cpu().numpy(), ref.values(bits, np.concatenate(small.k)))


@pytest.mark.parametrize("group", [1, 8])
def test_rows_past_32_bits_of_bytes(group):
    """Rows a gigabyte apart."""
    say("rows far apart", group)
    p = Pool(4, 2, 64, 64, [40], seed=2)
    ld, rows = 1 << 28, 6
    wide = torch.empty((rows, ld), device="cuda")
    heads = 2 * group
    near = torch.randn((rows, (heads + 4) * 64), device="cuda")
    wide[:, ld - near.shape[1]:] = near
    batch = p.batch(lens=[rows], starts=[0, rows], rows=rows)
    views = []
    for t in (near, wide[:, ld - near.shape[1]:]):
        k, v = (t[:, a * 64:(a + 2) * 64].unflatten(1, (2, 64)) for a in (heads, heads + 2))
        q8.cache_append(p.cache, batch, k, v)
        views.append((*q8.cache_read(p.cache, batch), *q8.attention(p.cache, batch, t[:, :heads * 64].unflatten(1, (heads, 64)))))
        p.cache.data.zero_()
    assert all(torch.equal(a, b) for a, b in zip(*views)) and (views[0][0] != 0).any()


@pytest.mark.parametrize("starts", [[0, 9, 4, 12], [-3, 5, 9, 12], [0, 5, 9, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, 3, 12], [13, 14, 15, 16]])
@pytest.mark.parametrize("lens", [[40, 40, 40], [-5, 2 ** 31 - 1, -2 ** 31], [0, 1, 2]])
@pytest.mark.parametrize("heads", [1, 2, 8])
def test_starts_that_make_no_sense_leave_the_attentions_guards(starts, lens, heads):
    """Rows are clipped to the call's arrays in both kernels (up to 32 query rows of a kv head, and more)."""
    say("guards", starts, lens, heads)
    p = Pool(4, 1, 64, 32, [40, 40, 40])
    p.cache.data.zero_()
    p.fill()
    out, lse = torch.full((32, heads, 64), 3.0, device="cuda"), torch.full((32, heads), 3.0, device="cuda")
    batch = p.batch(lens=lens, starts=starts, rows=12, max_rows=12)
    q8.attention(p.cache, batch, torch.ones((12, heads, 64), device="cuda"), out=out[10:22], lse=lse[10:22])
    torch.cuda.synchronize()
    for t in (out, lse):
        assert (t[:10] == 3).all() and (t[22:] == 3).all() and not torch.isnan(t).any()
    if starts == [13, 14, 15, 16]:  # no sequence has a row
        assert (out == 3).all() and (lse == 3).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_half_a_million_blocks_round_as_the_formulas_say(bits):
    """Blocks of 32 values on grids where quotients come near to half-integers: 262144 of keys and as many of values."""
    say("grids, half a million blocks", bits)
    rng = np.random.default_rng(90 + bits)
    n, dim = 32768, 256
    p = Pool(bits, 1, dim, 1024, [1])
    cache = q8.KVCache(bits, 1, dim, 1024, n // 1024)
    batch = q8.CacheBatch(cache, torch.arange(n // 1024, dtype=torch.int32, device="cuda")[None], _dev(np.array([n], np.int32)),
                          _dev(np.array([0, n], np.int32)), n)
    x = rng.standard_normal((n, 1, dim // 32, 32), dtype=np.float32)
    grid = rng.integers(0, 12, (n, 1, dim // 32, 1))
    x = np.where(grid < 10, (np.rint(x * 2.0 ** grid) / 2.0 ** grid).astype(np.float32), x)
    x = (x * rng.integers(1, 64, grid.shape) / 32).astype(np.float32)
    y = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.float32(9), np.float32(-9)))
    x, y = (t.reshape(n, 1, dim) for t in (x, y))
    q8.cache_append(cache, batch, _dev(x), _dev(y))
    for got, t in zip(q8.cache_read(cache, batch), (x, y)):
        assert np.array_equal(got.cpu().numpy().astype(np.float64), ref.values(bits, t))


@pytest.mark.parametrize("new", [1, 50])
def test_a_captured_call_without_a_workspace_of_the_callers(new):
    """Outputs and the workspace are the graph's own; replays over other lengths, the program's own calls between them."""
    say("captured, own workspace", new)
    p = Pool(4, 2, 128, 64, [2000, 300], seed=3).fill()
    lens = _dev(p.lens)
    batch = q8.CacheBatch(p.cache, _dev(p.table), lens, _dev(np.array([0, new, 2 * new], np.int32)), 2 * new, new)
    q = torch.randn((2 * new, 8, 128), device="cuda")
    q8.attention(p.cache, batch, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q8.attention(p.cache, batch, q)
    for n in ([2000, 300], [1999, 51], [100, 60], [2000, 300]):
        lens.copy_(_dev(np.array(n, np.int32)))
        want = q8.attention(p.cache, batch, q)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n
