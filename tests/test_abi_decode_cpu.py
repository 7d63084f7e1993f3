"""The C ABI of include/q8_decode.h without a GPU: exports, workspace sizes, and
every refusal before anything is enqueued (fake addresses; each call here fails
a check or is empty)."""
import ctypes
import os
import re

import pytest

import q8_projection_amd as q8
from q8_projection_amd.decode import _MoeLayerC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, MODE, ALIAS = 0, 1, 2, 3, 4, 5
BASE = 0x7f0000000000
MB = 1 << 20


def test_header_and_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "q8_decode.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(q8_\w+)\s*\(", text))
    assert names and all(n in q8.SIGNATURES and hasattr(q8.lib(), n) for n in names)


def layer(mode=2, experts=8, top_k=2, renorm=1, k=256, ff=128, router=BASE, wg=BASE + 16 * MB, wu=BASE + 32 * MB,
          wd=BASE + 48 * MB):
    return _MoeLayerC(mode, experts, top_k, renorm, k, ff, router, wg, wu, wd)


def moe(l, x=BASE + 64 * MB, rows=3, res=None, y=BASE + 80 * MB, ids=BASE + 96 * MB, gates=BASE + 97 * MB,
        ws=BASE + 112 * MB, wsb=1 << 30):
    return q8.lib().q8_moe(ctypes.addressof(l), x, rows, res, y, ids, gates, ws, wsb, None)


def experts(l, x=BASE + 64 * MB, rows=3, res=None, y=BASE + 80 * MB, ids=BASE + 96 * MB, gates=BASE + 97 * MB,
            ws=BASE + 112 * MB, wsb=1 << 30):
    return q8.lib().q8_moe_experts(ctypes.addressof(l), x, rows, ids, gates, res, y, ws, wsb, None)


def route(l, x=BASE + 64 * MB, rows=3, ids=BASE + 96 * MB, gates=BASE + 97 * MB, ws=BASE + 112 * MB, wsb=1 << 30):
    return q8.lib().q8_moe_route(ctypes.addressof(l), x, rows, ids, gates, ws, wsb, None)


def test_empty_calls_enqueue_nothing():
    l = layer()
    assert moe(l, rows=0) == OK and experts(l, rows=0) == OK and route(l, rows=0) == OK


def test_workspace_bytes():
    def size(rows, **kw):
        l = layer(**kw)
        return q8.lib().q8_moe_workspace_bytes(ctypes.addressof(l), rows)
    assert 0 < size(1) < size(64) == size(65) == size(1 << 20)
    assert size(4, mode=1) < size(4, mode=2)
    assert size(-1) == 0 and size(1, mode=3) == 0 and size(1, experts=0) == 0
    assert q8.lib().q8_moe_workspace_bytes(None, 1) == 0


@pytest.mark.parametrize("bad", [dict(experts=0), dict(experts=513), dict(experts=-1), dict(top_k=0), dict(top_k=9),
                                 dict(experts=64, top_k=17), dict(k=0), dict(k=96), dict(k=-64), dict(k=65536 + 64),
                                 dict(ff=32), dict(ff=1 << 40), dict(experts=512, k=65536, ff=65536)])
def test_bad_sizes(bad):
    for f in (moe, experts, route):
        assert f(layer(**bad)) == SHAPE, bad


def test_bad_rows_mode_and_workspace():
    for f in (moe, experts, route):
        assert f(layer(), rows=-1) == SHAPE
        assert f(layer(), rows=(1 << 20) + 1) == SHAPE
        assert f(layer(), rows=1 << 62) == SHAPE
        assert f(layer(mode=3)) == MODE and f(layer(mode=-1)) == MODE
        need = q8.lib().q8_moe_workspace_bytes(ctypes.addressof(layer()), 3)
        assert f(layer(), wsb=need - 1) == SHAPE
    assert q8.lib().q8_moe(None, BASE, 1, None, BASE, BASE, BASE, BASE, 1, None) == NULL


def test_null_pointers():
    for kw in (dict(x=None), dict(ids=None), dict(gates=None), dict(ws=None)):
        for f in (moe, experts, route):
            assert f(layer(), **kw) == NULL, kw
    assert moe(layer(), y=None) == NULL and experts(layer(), y=None) == NULL
    assert moe(layer(router=None)) == NULL and route(layer(router=None)) == NULL
    for kw in (dict(wg=None), dict(wu=None), dict(wd=None)):
        assert moe(layer(**kw)) == NULL and experts(layer(**kw)) == NULL


def test_alignment():
    for kw in (dict(x=BASE + 64 * MB + 8), dict(ids=BASE + 96 * MB + 2), dict(gates=BASE + 97 * MB + 1),
               dict(ws=BASE + 112 * MB + 8)):
        for f in (moe, experts, route):
            assert f(layer(), **kw) == ALIGN, kw
    assert moe(layer(router=BASE + 4)) == ALIGN and route(layer(router=BASE + 4)) == ALIGN
    for kw in (dict(wg=BASE + 16 * MB + 2), dict(wu=BASE + 32 * MB + 1), dict(wd=BASE + 48 * MB + 2)):
        assert moe(layer(**kw)) == ALIGN and experts(layer(**kw)) == ALIGN
    assert moe(layer(), y=BASE + 80 * MB + 2) == ALIGN and moe(layer(), res=BASE + 72 * MB + 1) == ALIGN


def test_overlaps():
    y, x, ids, gates, ws = BASE + 80 * MB, BASE + 64 * MB, BASE + 96 * MB, BASE + 97 * MB, BASE + 112 * MB
    for kw in (dict(y=x), dict(y=x + 16), dict(y=ids), dict(y=BASE + 16 * MB), dict(y=BASE + 32 * MB + 64),
               dict(y=BASE + 48 * MB), dict(y=ws), dict(ws=x), dict(ws=BASE + 48 * MB), dict(ws=ids - 256),
               dict(res=y + 4), dict(res=y - 4), dict(res=ws), dict(ids=x + 4, gates=gates)):
        assert moe(layer(), **kw) == ALIAS, kw
    for kw in (dict(ids=gates), dict(gates=x), dict(ids=BASE), dict(res=ids)):
        assert moe(layer(), **kw) == ALIAS, kw
    assert route(layer(), ids=gates + 4) == ALIAS
    assert experts(layer(), y=gates) == ALIAS


def sample(logits=BASE, ld=1000, rows=4, n=1000, t=BASE + 16 * MB, k=BASE + 17 * MB, p=BASE + 18 * MB, mp=BASE + 19 * MB,
           u=BASE + 20 * MB, idx=BASE + 21 * MB, prob=BASE + 22 * MB, ws=BASE + 32 * MB, wsb=1 << 30):
    return q8.lib().q8_sample(logits, ld, rows, n, t, k, p, mp, u, idx, prob, ws, wsb, None)


def test_sample_refusals():
    assert sample(rows=0) == OK
    size = q8.lib().q8_sample_workspace_bytes
    assert 0 < size(1, 1) <= size(4, 1000) < size(64, 151936)
    assert size(-1, 5) == size(1, 0) == size(1, 1 << 19) == size(65537, 1) == 0
    for kw in (dict(n=0), dict(n=-1), dict(n=1 << 19, ld=1 << 20), dict(ld=999), dict(rows=-1), dict(rows=65537),
               dict(rows=1 << 62), dict(ld=1 << 62), dict(wsb=size(4, 1000) - 1)):
        assert sample(**kw) == SHAPE, kw
    for kw in (dict(logits=None), dict(u=None), dict(idx=None), dict(ws=None)):
        assert sample(**kw) == NULL, kw
    for kw in (dict(logits=BASE + 2), dict(t=BASE + 16 * MB + 1), dict(k=BASE + 17 * MB + 2), dict(p=BASE + 18 * MB + 3),
               dict(mp=BASE + 19 * MB + 2), dict(u=BASE + 20 * MB + 1), dict(idx=BASE + 21 * MB + 2),
               dict(prob=BASE + 22 * MB + 2), dict(ws=BASE + 32 * MB + 8)):
        assert sample(**kw) == ALIGN, kw
    for kw in (dict(idx=BASE + 4 * 3999), dict(prob=BASE), dict(idx=BASE + 20 * MB), dict(prob=BASE + 21 * MB + 12),
               dict(ws=BASE), dict(ws=BASE + 21 * MB), dict(idx=BASE + 17 * MB + 4)):
        assert sample(**kw) == ALIAS, kw


def test_a_workspace_for_the_largest_call_serves_smaller_ones():
    """The bytes do not decrease with any size, so that a loop keeps one workspace."""
    lib = q8.lib()
    rows = [0, 1, 2, 3, 15, 16, 17, 20, 31, 32, 33, 40, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 1023, 1024, 1025, 5000]
    ns = [1, 64, 65, 4096, 4097, 9000, 30000, 65536, 65537, 131072, 151936, 262144, (1 << 19) - 1]
    for n in ns:
        sizes = [lib.q8_sample_workspace_bytes(r, n) for r in rows]
        assert sizes == sorted(sizes), n
    for r in rows:
        sizes = [lib.q8_sample_workspace_bytes(r, n) for n in ns]
        assert sizes == sorted(sizes), r
    for mode in (0, 1, 2):
        for experts, top_k, k, ff in ((1, 1, 64, 64), (8, 2, 256, 128), (64, 8, 2048, 1408), (512, 16, 128, 64), (3, 2, 16448, 64)):
            c = layer(mode=mode, experts=experts, top_k=top_k, k=k, ff=ff)
            sizes = [lib.q8_moe_workspace_bytes(ctypes.addressof(c), r) for r in range(70)]
            assert sizes[0] > 0 and sizes == sorted(sizes)
