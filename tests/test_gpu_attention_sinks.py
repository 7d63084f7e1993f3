"""Attention where one token has nearly all of the weight and adds next to nothing: the outputs are made of weights far
below the largest one.

Bound of the outputs.  A weight w_t goes to the matrix cores in two binary16 words of w_t / m, where the power of two m
follows the tiles of 32 tokens that a wave takes one after the other: the largest weight that a row has in a tile is
2^-1 or more of m's scale (a tile that is 12 powers of two below 2^11 lowers m, down to 2^-79 of a row's largest
weight: 54 nats), and in the tile of the row's largest weight 2^11 or more.  The words are off by 2^-22 w_t (half a step of
11 bits, twice) or, where the second ends on binary16's grid of 2^-24, by 2^-25: 2^-24 of the largest weight of the
tile, 2^-36 in the tile of the row's largest.  With everything else as in cache_reference.py,

    |out - ref| <= A (2 ez + 2^-20 + (T / 8 + 64) 2^-24) + sum_t e_t |v_t| / sum_t exp(z_t),
    e_t = 2^-24 max over t's tile of exp(z) (2^-36 of it in the tile of the largest z)

and the 2-norm of the errors is held to that of A (2 ez' + 2^-20 + sqrt(T) 2^-24) and of the e_t's share, added as squares.
(The tokens beside the heavy one have values of zero here, so that they take no part in either sum: 31 tokens of
thousands, whose weights have an error of 2^-36 of the heavy one's.)
"""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say
from test_gpu_cache import FORMS, Pool, _dev

pytestmark = pytest.mark.gpu


def sums(q, k, v, scale):
    """(out, lse, bound of out, usual error of out, bound of lse) of one f64 query [D] over k, v [T][D] from token 0 on."""
    d, n = k.shape[1], k.shape[0]
    z = scale * (k @ q)
    big = abs(scale) * (np.abs(k) @ np.abs(q)).max()
    e = np.exp(z - z.max())
    p = e / e.sum()
    tile = np.arange(n) // 32
    heaviest = np.maximum.reduceat(p, np.arange(0, n, 32))[tile]
    off = np.where(tile == z.argmax() // 32, 2.0 ** -36, 2.0 ** -24) * heaviest
    size = p @ np.abs(v)
    ez = big * (2.0 ** -21 + (d + 8) * 2.0 ** -24) + 8 * 2.0 ** -24 * (1 + np.abs(z).max())
    bound = size * (2 * ez + 2.0 ** -20 + (n / 8 + 64) * 2.0 ** -24) + off @ np.abs(v)
    usual = size * (2.0 ** -23 * (np.sqrt(d + 8) * big + 4 * (1 + np.abs(z).max())) + 2.0 ** -20 + np.sqrt(n) * 2.0 ** -24) + \
        np.sqrt(off ** 2 @ v ** 2)
    lse = z.max() + np.log(e.sum())
    return p @ v, lse, bound, usual, ez + (n / 8 + 64) * 2.0 ** -24 + 2.0 ** -23 * abs(lse)


def sinks(rng, n, dim, kv_heads, heavy, above):
    """Keys and values of n tokens, each at `heavy` scoring `above` nats more than those that its first dimension says nothing
    of, for queries of 8 in that dimension and a scale of 1 / sqrt(dim); values of zero in the heavy tokens' tiles."""
    k = rng.standard_normal((n, kv_heads, dim)).astype(np.float32)
    k[..., :32] = 0
    v = rng.uniform(0.5, 1.5, (n, kv_heads, dim)).astype(np.float32)
    for t, nats in zip(heavy, above):
        k[t] = 0
        k[t, :, 0] = nats * np.sqrt(dim) / 8
        v[t // 32 * 32:t // 32 * 32 + 32] = 0
    return k, v


def check(p, lens, news, heads, rng, sample=3):
    rows, dim, kv_heads = sum(news), p.dim, p.kv_heads
    q = (rng.standard_normal((rows, heads, dim)) * 0.5).astype(np.float32)
    q[..., 0] = 8
    begin = np.concatenate([[0], np.cumsum(news)])
    batch = p.batch(lens=lens, starts=begin, rows=rows, max_rows=max(news))
    out, lse = (t.cpu().numpy().astype(np.float64) for t in q8.attention(p.cache, batch, _dev(q)))
    for s in np.unique(np.r_[0, rng.integers(0, len(lens), 6)]):
        k, v = p.values(s)
        for r in np.unique(np.r_[0, news[s] - 1, rng.integers(0, news[s], sample)]):
            n = lens[s] - news[s] + r + 1
            err, usual = [], []
            for h in range(heads):
                kh = h // (heads // kv_heads)
                want, want_lse, bound, common, lse_bound = sums(q[begin[s] + r, h].astype(np.float64), k[:n, kh], v[:n, kh],
                                                                1 / np.sqrt(dim))
                err.append(np.abs(out[begin[s] + r, h] - want))
                usual.append(common)
                assert (err[-1] <= bound).all(), (s, r, h, (err[-1] / np.abs(want)).max())
                assert abs(lse[begin[s] + r, h] - want_lse) <= lse_bound, (s, r, h)
            assert np.linalg.norm(err) <= np.linalg.norm(usual), (s, r, np.linalg.norm(err) / np.linalg.norm(usual))


@pytest.mark.parametrize("above", [6, 10, 14, 20, 30, 45])
@pytest.mark.parametrize("bits,dim", FORMS)
def test_prompts_and_chunks_after_a_heavy_token(bits, dim, above):
    """Many rows: the first token takes all but exp(-above) thousands of the weight, or one in the middle does."""
    say("heavy, rows", bits, dim, above)
    rng = np.random.default_rng(above)
    lens, news = [1500, 900, 2300], [40, 900, 33]
    p = Pool(bits, 1, dim, 64, lens, seed=dim)
    p.k, p.v = map(list, zip(*(sinks(rng, n, dim, 1, [t], [above]) for n, t in zip(lens, (0, 0, 1000)))))
    check(p.fill(), lens, news, 4, rng)


@pytest.mark.parametrize("above", [6, 14, 20, 30, 45])
@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("new", [1, 3])
def test_tokens_after_a_heavy_one(bits, dim, above, new):
    """Few rows: a batch whose workgroups' waves take several tiles each."""
    say("heavy, few", bits, dim, above, new)
    rng = np.random.default_rng(above + new)
    lens = [1200 - 7 * i for i in range(40)]
    p = Pool(bits, 2, dim, 64, lens, seed=dim)
    p.k, p.v = map(list, zip(*(sinks(rng, n, dim, 2, [5 * i], [above]) for i, n in enumerate(lens))))
    check(p.fill(), lens, [new] * 40, 8, rng)


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 256)])
@pytest.mark.parametrize("new", [1, 50])
def test_heavy_tokens_of_many_weights(bits, dim, new):
    """Up and down, far apart and close together: each heavier than all before it, or lighter."""
    say("heavy, several", bits, dim, new)
    rng = np.random.default_rng(new)
    heavy, above = [3, 40, 300, 330, 700, 1000, 1400], [20, 30, 5, 40, 44, 12, 45]
    for order in (above, above[::-1]):
        lens = [2000] * 12
        p = Pool(bits, 2, dim, 64, lens, seed=dim)
        p.k, p.v = map(list, zip(*(sinks(rng, n, dim, 2, heavy, order) for n in lens)))
        check(p.fill(), lens, [new] * 12, 4, rng)


@pytest.mark.parametrize("bits,dim", [(4, 64), (4, 128), (8, 256)])
@pytest.mark.parametrize("new", [1, 40])
def test_heavy_tokens_beside_values_as_large_as_there_are(bits, dim, new):
    """A heavy token in every third tile: every wave's sums are lifted as far as they are, many parts of them joined."""
    say("heavy, large values", bits, dim, new)
    rng = np.random.default_rng(new)
    n, p = 9000, Pool(bits, 1, dim, 64, [9000], seed=dim)
    for above in (45, 70):  # (70: weights of 2^-101 of the largest, under what the words hold; the sums have to hold up)
        k, v = sinks(rng, n, dim, 1, list(range(7, n, 96)), [above] * 94)
        p.k, p.v = [k], [v * np.float32(4e4)]
        p.fill()
        if above == 45:
            check(p, [n], [new], 4, rng)
        q = torch.full((new, 4, dim), 0.25, device="cuda")
        q[..., 0] = 8
        out, lse = q8.attention(p.cache, p.batch(starts=[0, new], rows=new), q)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all() and (out >= 0).all()
