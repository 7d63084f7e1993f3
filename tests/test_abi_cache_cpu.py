"""The C ABI of include/q8_cache.h without a GPU: exports, sizes, and every refusal
before anything is enqueued (fake addresses; each call here fails a check or is
empty); and the reference's own layout and rounding."""
import ctypes
import os
import re

import numpy as np
import pytest

import cache_reference as ref
import q8_projection_amd as q8
from q8_projection_amd.cache import _BatchC, _CacheC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, MODE, ALIAS = 0, 1, 2, 3, 4, 5
BASE = 0x7f0000000000
GB = 1 << 30


def test_header_and_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q8_cache.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(q8_\w+)\s*\(", text))
    assert len(names) == 5 and all(n in q8.SIGNATURES and hasattr(q8.lib(), n) for n in names)


def cache(bits=4, kv_heads=4, head_dim=128, page_tokens=64, pages=100, data=BASE):
    return _CacheC(bits, kv_heads, head_dim, page_tokens, pages, data)


def batch(sequences=3, table_ld=8, table=BASE + 10 * GB, lens=BASE + 11 * GB, starts=BASE + 12 * GB, rows=20, max_rows=9):
    return _BatchC(sequences, table_ld, table, lens, starts, rows, max_rows)


def at(c):
    return None if c is None else ctypes.addressof(c)


def append(c, b, k=BASE + 20 * GB, k_ld=512, v=BASE + 21 * GB, v_ld=512):
    return q8.lib().q8_cache_append(at(c), at(b), k, k_ld, v, v_ld, None)


def read(c, b, k=BASE + 20 * GB, v=BASE + 21 * GB):
    return q8.lib().q8_cache_read(at(c), at(b), k, v, None)


def attend(c, b, q=BASE + 20 * GB, q_ld=1024, heads=8, window=0, out=BASE + 22 * GB, lse=BASE + 23 * GB, ws=BASE + 30 * GB,
           wsb=1 << 40):
    return q8.lib().q8_attention(at(c), at(b), q, q_ld, heads, 0.1, window, out, lse, ws, wsb, None)


def size(c, b, heads):
    return q8.lib().q8_attention_workspace_bytes(at(c), at(b), heads)


CALLS = (append, read, attend)


def test_page_bytes():
    for bits, d in ((4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)):
        assert q8.cache_page_bytes(bits, 3, d, 128) == 3 * 4 * ref.tile_parts(bits, d)[-1]
        assert ref.tile_parts(bits, d)[-1] == 2 * 32 * (d * bits // 8 + d // 32 * 2)
    assert q8.cache_page_bytes(4, 8, 128, 32) == 8 * 4608
    assert q8.lib().q8_cache_page_bytes(None) == 0


BAD_FORMATS = [dict(kv_heads=0), dict(kv_heads=257), dict(kv_heads=-1), dict(head_dim=0), dict(head_dim=96),
               dict(head_dim=512), dict(page_tokens=16), dict(page_tokens=48), dict(page_tokens=8192), dict(page_tokens=0),
               dict(page_tokens=-64), dict(page_tokens=-2 ** 31)]


@pytest.mark.parametrize("bad", BAD_FORMATS)
def test_bad_formats(bad):
    c = cache(**bad)
    assert all(f(c, batch()) == SHAPE for f in CALLS)
    assert q8.lib().q8_cache_page_bytes(at(c)) == 0
    assert size(c, batch(), 8) == 0


def test_bad_bits_and_pages():
    for bits in (0, 3, 5, 16, -4):
        assert all(f(cache(bits=bits), batch()) == MODE for f in CALLS)
        assert q8.cache_page_bytes(bits, 4, 128, 64) == 0
    for pages in (0, -1, 1 << 31, 1 << 62):
        assert all(f(cache(pages=pages), batch()) == SHAPE for f in CALLS)


@pytest.mark.parametrize("bad", [dict(sequences=-1), dict(sequences=65537), dict(table_ld=0), dict(table_ld=-1),
                                 dict(table_ld=(1 << 24) + 1), dict(table_ld=1 << 60), dict(rows=-1),
                                 dict(rows=(1 << 20) + 1), dict(rows=1 << 62), dict(max_rows=0), dict(max_rows=-1),
                                 dict(starts=None, rows=4), dict(starts=None, rows=2),
                                 dict(sequences=65536, rows=1 << 20, max_rows=1 << 62)])
def test_bad_batches(bad):
    assert all(f(cache(), batch(**bad)) == SHAPE for f in CALLS), bad
    assert size(cache(), batch(**bad), 8) == 0


def test_nothing_to_do_enqueues_nothing():
    for f in CALLS:
        assert f(cache(), batch(rows=0)) == OK
        assert f(cache(), batch(sequences=0)) == OK
        assert f(cache(), batch(sequences=0, rows=0, starts=None)) == OK
    assert size(cache(), batch(), 8) > 0


def test_null_pointers():
    for f in CALLS:
        assert f(None, batch()) == NULL and f(cache(), None) == NULL
        assert f(cache(data=None), batch()) == NULL
        assert f(cache(), batch(table=None)) == NULL and f(cache(), batch(lens=None)) == NULL
    for f in (append, read):
        assert f(cache(), batch(), k=None) == NULL and f(cache(), batch(), v=None) == NULL
    for kw in (dict(q=None), dict(out=None), dict(ws=None)):
        assert attend(cache(), batch(), **kw) == NULL


def test_strides_heads_window_and_workspace():
    for f, name in ((append, "k_ld"), (append, "v_ld"), (attend, "q_ld")):
        for bad in (0, -4, 508, 514, 1 << 62):
            assert f(cache(), batch(), **{name: bad}) == SHAPE
    assert attend(cache(), batch(), q_ld=1020) == SHAPE
    for heads in (0, -4, 6, 4100, 1 << 40):
        assert attend(cache(), batch(), heads=heads, q_ld=1 << 20) == SHAPE
    for window in (-1, 1 << 31, 1 << 62):
        assert attend(cache(), batch(), window=window) == SHAPE
    need = size(cache(), batch(), 8)
    assert attend(cache(), batch(), wsb=need - 1) == SHAPE


def test_alignment():
    for f in CALLS:
        assert f(cache(data=BASE + 8), batch()) == ALIGN
        for name in ("table", "lens", "starts"):
            assert f(cache(), batch(**{name: BASE + 10 * GB + 2})) == ALIGN
    for f in (append, read):
        assert f(cache(), batch(), k=BASE + 20 * GB + 4) == ALIGN and f(cache(), batch(), v=BASE + 21 * GB + 8) == ALIGN
    for kw in (dict(q=BASE + 20 * GB + 4), dict(out=BASE + 22 * GB + 8), dict(lse=BASE + 23 * GB + 2), dict(ws=BASE + 30 * GB + 8)):
        assert attend(cache(), batch(), **kw) == ALIGN


def test_overlaps():
    size = 100 * q8.cache_page_bytes(4, 4, 128, 64)
    table, lens, starts = BASE + 10 * GB, BASE + 11 * GB, BASE + 12 * GB
    for name in ("k", "v"):
        assert append(cache(), batch(), **{name: BASE + size - 16}) == ALIAS
        assert read(cache(), batch(), **{name: BASE + size - 16}) == ALIAS
        for p in (table, lens, starts):
            assert read(cache(), batch(), **{name: p}) == ALIAS
    assert read(cache(), batch(), k=BASE + 20 * GB, v=BASE + 20 * GB + 16) == ALIAS
    assert append(cache(data=table - 16), batch()) == ALIAS
    q, out, lse, ws = BASE + 20 * GB, BASE + 22 * GB, BASE + 23 * GB, BASE + 30 * GB
    for kw in (dict(out=q), dict(out=q + 20 * 4096 - 16), dict(out=BASE), dict(out=table), dict(out=lens), dict(out=starts),
               dict(lse=out), dict(lse=q + 4), dict(lse=ws), dict(ws=q), dict(ws=out), dict(ws=BASE), dict(ws=lens),
               dict(lse=starts)):
        assert attend(cache(), batch(), **kw) == ALIAS, kw


def test_workspace_for_the_largest_call_serves_smaller_ones():
    for bits, d in ((4, 128), (8, 64), (4, 256)):
        c = cache(bits=bits, head_dim=d)
        for heads in (4, 8, 32, 128):
            rows = [size(c, batch(sequences=3, rows=n, max_rows=n), heads) for n in (1, 2, 3, 4, 5, 8, 9, 17, 33, 64, 65, 100, 1000, 5000)]
            assert rows[0] > 0 and rows == sorted(rows), (d, heads, rows)
            seqs = [size(c, batch(sequences=n, rows=n, max_rows=1, starts=None), heads) for n in (1, 2, 7, 8, 9, 64, 65, 500, 65536)]
            assert seqs == sorted(seqs), (d, heads, seqs)
            assert size(c, batch(sequences=3, rows=300, max_rows=100), heads) <= size(c, batch(sequences=4, rows=400, max_rows=100), heads)


def test_reference_rounds_as_the_formulas_say():
    """Values off by at most d / 2, scales no longer than they have to be, binary16 values."""
    rng = np.random.default_rng(5)
    for bits, steps in ((4, 15), (8, 127)):
        x = (rng.standard_normal((400, 64)) * 10.0 ** rng.integers(-6, 4, (400, 1))).astype(np.float32)
        x[:40] = np.abs(x[:40])
        x[40:80, 32:] = 0
        _, d, _ = ref.quantize(bits, x)
        got = ref.values(bits, x)
        b, g = x.reshape(400, 2, 32).astype(np.float64), got.reshape(400, 2, 32)
        assert (np.abs(b - g) <= d[..., None] / 2).all()
        assert (got == got.astype(np.float16)).all()
        lo, hi = np.minimum(b.min(-1), 0), np.maximum(b.max(-1), 0)
        span = hi - lo if bits == 4 else np.maximum(hi, -lo)
        s = ref.scales(bits)
        below = s[np.maximum(np.searchsorted(s, d) - 1, 0)]
        assert (d * steps >= span).all() and ((below * steps < span) | (d == 0)).all()
