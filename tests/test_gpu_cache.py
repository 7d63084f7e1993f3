"""The key/value cache on the GPU: codes and words bit for bit against the formulas
and the layout, tokens that are not a call's left as they were."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import q8_projection_amd as q8
from helpers import say

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def normal(rng, *shape):
    x = rng.standard_normal(shape).astype(np.float32)
    x[..., 3::17] *= 8  # channels that stand out
    return x


def same(got, bits, x):
    """Every value read back is the one that the formulas give for x."""
    got, want = got.cpu().numpy().astype(np.float64), ref.values(bits, x)
    off = np.argwhere(got != want)
    assert not len(off), (len(off), off[0], got[tuple(off[0])], want[tuple(off[0])])


class Pool:
    """A pool of garbage, sequences with pages of their own in a shuffled order, and what they hold."""

    def __init__(self, bits, kv_heads, dim, page, lens, entries=None, seed=1):
        self.rng = rng = np.random.default_rng(seed)
        self.bits, self.kv_heads, self.dim, self.page = bits, kv_heads, dim, page
        self.entries = entries or max(1, *(-(-n // page) for n in lens))
        need = [min(-(-n // page), self.entries) for n in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(lens), self.entries), -7, np.int32)
        first = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[first:first + n]
            first += n
        self.lens = np.array(lens, np.int32)
        size = q8.cache_page_bytes(bits, kv_heads, dim, page)
        self.before = rng.integers(0, 256, (pages, size), dtype=np.uint8)
        self.cache = q8.KVCache(bits, kv_heads, dim, page, _dev(self.before))
        self.k = [normal(rng, n, kv_heads, dim) for n in lens]
        self.v = [normal(rng, n, kv_heads, dim) for n in lens]

    def batch(self, lens=None, starts=None, rows=None, max_rows=None):
        return q8.CacheBatch(self.cache, _dev(self.table), _dev(self.lens if lens is None else np.array(lens, np.int32)),
                             None if starts is None else _dev(np.array(starts, np.int32)), rows, max_rows)

    def fill(self):
        """All sequences written with one call."""
        if self.lens.sum():
            starts = np.concatenate([[0], np.cumsum(self.lens)])
            q8.cache_append(self.cache, self.batch(starts=starts, rows=int(starts[-1]), max_rows=int(self.lens.max())),
                            _dev(np.concatenate(self.k)), _dev(np.concatenate(self.v)))
        return self

    def values(self, s):
        return ref.values(self.bits, self.k[s]), ref.values(self.bits, self.v[s])

    def packed(self, lens):
        """The pool's bytes after the first lens[s] tokens of each sequence were written, from the layout's formulas."""
        want = self.before.copy()
        d, size = self.dim, ref.tile_parts(self.bits, self.dim)[-1]
        tiles = want.reshape(want.shape[0], self.kv_heads, self.page // 32, size)
        for s, n in enumerate(lens):
            for t0 in range(0, n, 32):
                here = min(32, n - t0)
                for h in range(self.kv_heads):
                    k, v = np.zeros((32, d), np.float32), np.zeros((32, d), np.float32)
                    k[:here], v[:here] = self.k[s][t0:t0 + here, h], self.v[s][t0:t0 + here, h]
                    tile = np.zeros(size, np.uint8)
                    ref.pack(self.bits, k, v, tile)
                    dst = tiles[self.table[s, t0 // self.page], h, t0 % self.page // 32]
                    mask = np.zeros(size, np.uint8)
                    ref_mask(self.bits, d, here, mask)
                    dst[:] = (dst & ~mask) | (tile & mask)
        return want


def ref_mask(bits, d, tokens, mask):
    """Bits of a tile that the first `tokens` tokens own."""
    kc, kw, vc, vw, _ = ref.tile_parts(bits, d)
    for t in range(tokens):
        a, b, i = t // 8, t % 4, t % 8 // 4
        mask[kc + t * d * bits // 8:kc + (t + 1) * d * bits // 8] = 255
        for dim in range(d):
            w, c = dim // 16, dim % 16
            if bits == 4:
                mask[vc + ((((w // 4 * 4 + a) * 16 + c) * 4 + w % 4) * 8 + t % 8) // 2] |= 15 << 4 * (t % 2)
            else:
                mask[vc + ((((w // 2 * 4 + a) * 16 + c) * 2 + w % 2) * 4 + b) * 2 + i] = 255
        for blk in range(d // 32):
            at = kw + 2 * (((a * 4 + b) * (d // 32) + blk) * 2 + i)
            mask[at:at + 2] = 255
            at = vw + 2 * (((blk * 4 + a) * 4 + b) * 2 + i)
            mask[at:at + 2] = 255


FORMS = [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)]


@pytest.mark.parametrize("bits,dim", FORMS)
def test_bytes_of_the_layout(bits, dim):
    """The pool's every byte after a prompt and single tokens: written ones by the formulas, others untouched."""
    say("layout", bits, dim)
    p = Pool(bits, 2, dim, 64, [41, 70, 1], entries=3)
    first = [37, 61, 0]
    starts = np.concatenate([[0], np.cumsum(first)])
    q8.cache_append(p.cache, p.batch(lens=first, starts=starts, rows=int(starts[-1]), max_rows=61),
                    _dev(np.concatenate([x[:n] for x, n in zip(p.k, first)])),
                    _dev(np.concatenate([x[:n] for x, n in zip(p.v, first)])))
    assert np.array_equal(p.cache.data.cpu().numpy(), p.packed(first))
    lens = list(first)
    while lens != [41, 70, 1]:  # a token at a time, sequences that are done as empty slots
        go = [n < m for n, m in zip(lens, [41, 70, 1])]
        lens = [n + g for n, g in zip(lens, go)]
        row = lambda x: np.stack([x[s][lens[s] - 1] if go[s] else np.full((2, dim), 9, np.float32) for s in range(3)])  # noqa: E731
        q8.cache_append(p.cache, p.batch(lens=[n if g else 0 for n, g in zip(lens, go)]), _dev(row(p.k)), _dev(row(p.v)))
    assert np.array_equal(p.cache.data.cpu().numpy(), p.packed(lens))


@pytest.mark.parametrize("bits,dim", FORMS)
@pytest.mark.parametrize("page", [32, 256])
def test_written_and_read_back(bits, dim, page):
    say("append and read", bits, dim, page)
    lens = [0, 1, 31, 32, 33, 129, 300, 7]
    p = Pool(bits, 3, dim, page, lens, seed=dim + page).fill()
    starts = np.concatenate([[0], np.cumsum(lens)])
    rows = int(starts[-1])
    k, v = q8.cache_read(p.cache, p.batch(starts=starts, rows=rows, max_rows=300))
    for got, x in ((k, p.k), (v, p.v)):
        want = ref.values(bits, np.concatenate(x))
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want)
    # the last rows alone, and more than a sequence has
    n = [min(m, 5) for m in lens]
    starts = np.concatenate([[0], np.cumsum(n)])
    k, v = q8.cache_read(p.cache, p.batch(starts=starts, rows=int(starts[-1]), max_rows=5))
    assert np.array_equal(k.cpu().numpy(), ref.values(bits, np.concatenate([x[len(x) - m:] for x, m in zip(p.k, n)])))
    k, v = q8.cache_read(p.cache, p.batch(starts=np.arange(9) * 40, rows=320, max_rows=40))
    for got, x in ((k, p.k), (v, p.v)):
        for s, m in enumerate(lens):
            want = np.zeros((40, 3, dim))
            here = min(m, 40)
            if here:
                want[40 - here:] = ref.values(bits, x[s][m - here:])
            assert np.array_equal(got[40 * s:40 * s + 40].cpu().numpy(), want), s


def specials(dim):
    """Blocks that meet the formulas' corners, [rows][dim]."""
    rows = []
    for base in (np.zeros(32), np.full(32, 2.5), np.full(32, -2.5), np.linspace(0, 15, 32), np.linspace(-7.5, 7.5, 32),
                 np.linspace(-15, 0, 32), np.linspace(-127, 127, 32), np.r_[np.zeros(31), 1], np.r_[np.zeros(31), -1],
                 np.r_[0.5, 1.5, 2.5, 3.5, -0.5, -1.5, -2.5, -7.5, np.zeros(23), 7.5],
                 np.r_[np.arange(30) / 2, 0, 15], np.r_[np.arange(30) + 0.5, -127, 127]):
        for factor in (1.0, 2.0 ** -10, 2.0 ** -17, 2.0 ** -19, 1.5 * 2.0 ** -19, 2.0 ** -22, 2.0 ** -40, 1e-39, 1.03125, 1.0313,
                       1.125, 1.1251, 300.0, 4352.0, 1e5, 1e30, 3e38 / 127):
            rows.append(base * factor)
    x = np.array(rows, np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(-np.inf))])
    x = x[np.isfinite(x).all(1)]
    return np.tile(x, (1, dim // 32))


@pytest.mark.parametrize("bits,dim", [(4, 64), (8, 64), (4, 256), (8, 128)])
def test_corners_of_the_formulas(bits, dim):
    say("corners", bits, dim)
    x = specials(dim)[:, None]
    y = np.ascontiguousarray(x[::-1])
    p = Pool(bits, 1, dim, 64, [len(x)])
    batch = p.batch(starts=[0, len(x)], rows=len(x))
    q8.cache_append(p.cache, batch, _dev(x), _dev(y))
    k, v = q8.cache_read(p.cache, batch)
    same(k, bits, x)
    same(v, bits, y)


@pytest.mark.parametrize("bits", [4, 8])
def test_many_blocks_round_as_the_formulas_say(bits):
    """Half a million blocks on grids where quotients come near to half-integers."""
    say("grids", bits)
    rng = np.random.default_rng(9)
    n = 8192
    x = rng.standard_normal((n, 1, 64)).astype(np.float32)
    grid = rng.integers(0, 12, (n, 1, 1))
    x = np.where(grid < 10, (np.rint(x * 2.0 ** grid) / 2.0 ** grid).astype(np.float32), x)
    x = (x * rng.integers(1, 64, (n, 1, 1)) / 32).astype(np.float32)
    y = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.float32(9), np.float32(-9)))
    p = Pool(bits, 1, 64, 1024, [n])
    batch = p.batch(starts=[0, n], rows=n)
    q8.cache_append(p.cache, batch, _dev(x), _dev(y))
    k, v = q8.cache_read(p.cache, batch)
    same(k, bits, x)
    same(v, bits, y)


@pytest.mark.parametrize("bits", [4, 8])
def test_views_of_a_wider_buffer_and_outputs_given(bits):
    p = Pool(bits, 2, 128, 32, [40, 9], seed=3)
    rows, wide = 49, 5 * 2 * 128
    fused = torch.full((rows, wide), float("nan"), device="cuda")
    k, v = fused[:, 256:512].unflatten(1, (2, 128)), fused[:, 1024:].unflatten(1, (2, 128))
    k.copy_(_dev(np.concatenate(p.k)))
    v.copy_(_dev(np.concatenate(p.v)))
    batch = p.batch(starts=[0, 40, 49], rows=rows, max_rows=40)
    q8.cache_append(p.cache, batch, k, v)
    out = torch.empty((rows, 2, 128), device="cuda"), torch.empty((rows, 2, 128), device="cuda")
    got = q8.cache_read(p.cache, batch, *out)
    assert got[0] is out[0] and got[1] is out[1]
    for o, x in zip(out, (p.k, p.v)):
        assert np.array_equal(o.cpu().numpy(), ref.values(bits, np.concatenate(x)))


@pytest.mark.parametrize("bits,dim", [(4, 128), (8, 64)])
def test_tokens_that_are_none(bits, dim):
    """Pages outside the pool, tokens past the table, rows behind the last sequence, more rows than max_rows."""
    say("no tokens", bits, dim)
    p = Pool(bits, 2, dim, 32, [100, 64, 20], entries=4)
    p.table[0, 1] = p.cache.pages  # the first that the pool does not have
    p.table[1, 0] = -1
    lens = [100, 64 + 128, 20]      # the second sequence's last tokens lie past the table
    starts = [0, 100, 100 + 192, 100 + 192 + 20]
    rows = starts[-1] + 6
    k = normal(p.rng, rows, 2, dim)
    v = normal(p.rng, rows, 2, dim)
    p.table[1, 2:] = [p.cache.pages + 5, 2 ** 31 - 1]
    batch = p.batch(lens=lens, starts=starts, rows=rows, max_rows=192)
    q8.cache_append(p.cache, batch, _dev(k), _dev(v))
    out = torch.full((rows, 2, dim), 5.0, device="cuda"), torch.full((rows, 2, dim), 5.0, device="cuda")
    q8.cache_read(p.cache, batch, *out)
    for got, x in zip(out, (k, v)):
        want = ref.values(bits, x)
        want[32:64] = 0                       # sequence 0's second page
        want[100:132] = 0                     # sequence 1's first page
        want[100 + 64:292] = 0                # its third, fourth and what lies past the table
        want[312:] = 5                        # rows of no sequence
        assert np.array_equal(got.cpu().numpy(), want)
    # a sequence of more rows than max_rows: the first max_rows are served
    out = torch.full((rows, 2, dim), 5.0, device="cuda"), torch.full((rows, 2, dim), 5.0, device="cuda")
    q8.cache_read(p.cache, p.batch(lens=lens, starts=starts, rows=rows, max_rows=7), *out)
    want = ref.values(bits, k)
    got = out[0].cpu().numpy()
    assert np.array_equal(got[:7], want[:7]) and (got[7:100] == 5).all()
    assert np.array_equal(got[292:299], want[292:299]) and (got[299:] == 5).all()


@pytest.mark.parametrize("starts", [[0, 9, 4, 12], [-3, 5, 9, 12], [0, 5, 9, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, 3, 12], [13, 14, 15, 16]])
def test_starts_that_make_no_sense_reach_no_other_memory(starts):
    """Rows are clipped to the call's arrays; what the guard rows around them hold stays."""
    say("starts", starts)
    p = Pool(4, 1, 64, 32, [40, 40, 40]).fill()
    guard = torch.full((2, 12 + 20, 1, 64), 3.0, device="cuda")
    batch = p.batch(starts=starts, rows=12, max_rows=12)
    for lens in ([40, 40, 40], [-5, 2 ** 31 - 1, -2 ** 31], [0, 1, 2]):
        batch = p.batch(lens=lens, starts=starts, rows=12, max_rows=12)
        q8.cache_read(p.cache, batch, guard[0, 10:22], guard[1, 10:22])
        q8.cache_append(p.cache, batch, torch.ones((12, 1, 64), device="cuda"), torch.ones((12, 1, 64), device="cuda"))
        q = torch.ones((12, 2, 64), device="cuda")
        out, lse = q8.attention(p.cache, batch, q)
        torch.cuda.synchronize()
        assert (guard[:, :10] == 3).all() and (guard[:, 22:] == 3).all()


def test_refusals_of_the_wrappers():
    p = Pool(4, 2, 64, 32, [40, 9])
    batch = p.batch()
    ok = torch.zeros((2, 2, 64), device="cuda")
    for bad in (ok.double(), ok.cpu(), ok[:1], torch.zeros((2, 3, 64), device="cuda"), torch.zeros((2, 2, 128), device="cuda")[..., ::2],
                torch.zeros((2, 64, 2), device="cuda").transpose(1, 2), ok.view(2, 128), None):
        with pytest.raises(ValueError):
            q8.cache_append(p.cache, batch, bad, ok)
        with pytest.raises(ValueError):
            q8.cache_append(p.cache, batch, ok, bad)
        with pytest.raises(ValueError):
            q8.attention(p.cache, batch, bad if bad is not None and bad.shape[1:2] != (3,) else None)
    for make in (lambda: q8.KVCache(5, 2, 64, 32, p.cache.data), lambda: q8.KVCache(4, 3, 64, 32, p.cache.data),
                 lambda: q8.KVCache(4, 2, 64, 32, p.cache.data.cpu()), lambda: q8.KVCache(4, 2, 96, 32, 4),
                 lambda: q8.KVCache(4, 2, 64, 32, 0), lambda: q8.KVCache(4, 2, 64, 48, 4),
                 lambda: q8.CacheBatch(p.cache, _dev(p.table).long(), _dev(p.lens)),
                 lambda: q8.CacheBatch(p.cache, _dev(p.table), _dev(p.lens[:1])),
                 lambda: q8.CacheBatch(p.cache, _dev(p.table), _dev(p.lens), rows=3),
                 lambda: q8.CacheBatch(p.cache, _dev(p.table), _dev(p.lens), starts=_dev(p.lens), rows=3),
                 lambda: q8.CacheBatch(p.cache, _dev(p.table), _dev(p.lens), starts=_dev(np.array([0, 1, 2], np.int32)))):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(ValueError):
        q8.cache_read(p.cache, batch, k=torch.empty((2, 2, 32), device="cuda"))
    with pytest.raises(ValueError):
        q8.attention(p.cache, batch, ok, workspace=torch.zeros(16, device="cuda"))
    with pytest.raises(q8.Q8Error):
        q8.attention(p.cache, batch, ok, workspace=torch.zeros(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(q8.Q8Error):
        q8.attention(p.cache, batch, torch.zeros((2, 3, 64), device="cuda"))
    with pytest.raises(q8.Q8Error):
        q8.attention(p.cache, batch, ok, window=-1, workspace=q8.attention_workspace(p.cache, batch, 2))
