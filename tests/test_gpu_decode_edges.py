"""The decode-step calls at the ends of what they take: the largest sizes, addresses past
32 bits, the least alignment, logits as a bf16 head gives them, calls at once and
captured forks.  Tolerances are those of test_gpu_moe.py and test_gpu_sample.py.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import q8_projection_amd as q8
import sample_reference
from helpers import gate, say
from test_gpu_moe import _dev, inputs, make
from test_gpu_moe_paths import check as check_layer
from test_gpu_sample import KINDS, check, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows,experts,top_k,k,ff", [(1, 1, 1, 65536, 64), (3, 2, 1, 65536, 64), (6, 1, 1, 65536, 64),
                                                     (1, 1, 1, 64, 65536), (3, 2, 1, 64, 65536), (6, 1, 1, 64, 65536)])
def test_the_longest_rows_and_columns(mode, rows, experts, top_k, k, ff):
    check_layer(mode, rows, experts, top_k, k, ff)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_the_most_pairs_on_the_matrix_cores(mode):
    """64 rows of 16 choices among 256 (in the f32 mode, few enough for the vector kernels
    too) and 128 experts."""
    for experts in (256, 128):
        check_layer(mode, 64, experts, 16, 64, 64, renormalize=False)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows", [2, 9, 64])
def test_experts_past_32_bits(mode, rows):
    """The last of 512 experts whose matrices take 4.6 GB each (all three in one buffer),
    the others zero."""
    experts, k, ff = 512, 2048, 4096
    say("experts past 32 bits", mode, rows)
    _, (blocks, _, _), _ = make(mode, 1, 1, k, ff)
    w = torch.zeros((experts, ff, k // 32 * 34), dtype=torch.uint8, device="cuda")
    w[-1] = _dev(blocks[0])
    down = w.view(experts, k, ff // 32 * 34)
    layer = q8.MoeLayer(mode, w, w, down, k, ff, 16)
    x, res = inputs(rows, k, 3100 + rows)
    ids = np.full((rows, 16), -1, np.int32)
    ids[:, 15] = experts - 1
    ids[0, :] = np.arange(16)
    gates = np.random.default_rng(rows).random((rows, 16)).astype(np.float32)
    y = q8.moe_experts(layer, _dev(x), _dev(ids), _dev(gates), residual=_dev(res))
    torch.cuda.synchronize()
    only = np.where(ids == experts - 1, 0, -1)
    last = blocks.reshape(1, ff, -1)
    r, a = ref.experts(mode, last, last, blocks.reshape(1, k, -1), k, ff, x, only, gates, res)
    gate(y.cpu().numpy(), r, a, f"{mode} {rows}, the last of {experts}")


def offset(t, by):
    """The same values `by` bytes past an address that is a multiple of 256."""
    raw = torch.zeros(t.numel() * t.element_size() + 256, dtype=torch.uint8, device="cuda")
    raw[by:by + t.numel() * t.element_size()] = t.contiguous().view(-1).view(torch.uint8)
    return raw[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_the_least_alignment(mode, rows):
    """What may lie at any multiple of 4 bytes (16 for x, the router and the workspace) does."""
    experts, top_k, k, ff = 6, 2, 320, 192
    layer, (wg, wu, wd), router = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 3300 + rows)
    want = q8.moe(layer, _dev(x), residual=_dev(res))
    odd = q8.MoeLayer(mode, offset(_dev(wg), 4), offset(_dev(wu), 12), offset(_dev(wd), 20), k, ff, top_k,
                      router=offset(_dev(router), 16))
    out = offset(torch.zeros((rows, k), device="cuda"), 4)
    ids = offset(torch.zeros((rows, top_k), dtype=torch.int32, device="cuda"), 12)
    gates = offset(torch.zeros((rows, top_k), device="cuda"), 20)
    work = offset(torch.zeros(odd.workspace_bytes(rows), dtype=torch.uint8, device="cuda"), 16)
    for _ in range(2):
        q8.moe(odd, offset(_dev(x), 16), residual=offset(_dev(res), 28), out=out, ids=ids, gates=gates, workspace=work)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(ids, want[1]) and torch.equal(gates, want[2])


@pytest.mark.parametrize("mode", ["f32", "i8x2"])
@pytest.mark.parametrize("rows", [64, 130])
def test_in_place_over_slices_and_shared_tiles(mode, rows):
    layer, _, _ = make(mode, 6, 3, 512, 256)
    x, res = inputs(rows, 512, 3400 + rows)
    xd, rd = _dev(x), _dev(res)
    want = q8.moe(layer, xd, residual=rd)[0]
    for _ in range(3):
        y = rd.clone()
        q8.moe(layer, xd, residual=y, out=y)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_calls_at_once_on_two_streams():
    """Two streams, a workspace each, many calls in flight: the results of calls alone."""
    rows, n = 48, 32003
    layer, _, _ = make("i8x2", 16, 4, 512, 256)
    xs = [_dev(inputs(rows, 512, 3500 + i)[0]) for i in range(2)]
    logits = [torch.from_numpy(logits_of(rows, n, 3600 + i)).cuda() for i in range(2)]
    u, p = torch.rand(rows, device="cuda"), torch.full((rows,), 0.9, device="cuda")
    want = [q8.moe(layer, x) + q8.sample(l, u, top_p=p) for x, l in zip(xs, logits)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [layer.workspace(rows) for _ in range(2)]
    scratch = [torch.empty(q8.sample_workspace_bytes(rows, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(q8.moe(layer, xs[i], workspace=work[i], stream=s) +
                          q8.sample(logits[i], u, top_p=p, workspace=scratch[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_a_captured_fork_that_allocates():
    """Calls on a stream forked inside a capture, outputs and workspaces made by the calls."""
    rows, n = 5, 20011
    layer, _, _ = make("i8x2", 8, 2, 256, 128)
    xs = [_dev(inputs(rows, 256, 3700 + i)[0]) for i in range(3)]
    ls = [torch.from_numpy(logits_of(rows, n, 3800 + i)).cuda() for i in range(3)]
    u, p = torch.rand(rows, device="cuda"), torch.full((rows,), 0.8, device="cuda")
    want = [q8.moe(layer, x) + q8.sample(l, u, top_p=p) for x, l in zip(xs, ls)]
    x, l, side = xs[0].clone(), ls[0].clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        drawn = q8.sample(l, u, top_p=p, stream=side)
        y = q8.moe(layer, x)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for i in range(3):
            x.copy_(xs[i])
            l.copy_(ls[i])
            graph.replay()
            eager = q8.moe(layer, xs[i]) + q8.sample(ls[i], u, top_p=p)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(y + drawn, want[i]))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[i]))


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,n", [(2, 151936), (6, 32003)])
def test_logits_of_a_bf16_head(kind, rows, n):
    """Logits on bf16's grid: thousands of equal ones where the prefixes end."""
    say("bf16 logits", kind, rows, n)
    l = torch.from_numpy(logits_of(rows, n, 41 + n)).bfloat16().float().numpy()
    for u in (None, 0.97):
        check(l, u=u, what=(kind, u), **KINDS[kind])


def test_parameters_at_the_ends_of_their_types():
    l = logits_of(6, 9001, 47)
    tiny, last = np.float32(1e-45), np.float32(1 - 2.0 ** -24)
    for kw in (dict(min_p=tiny), dict(min_p=last), dict(top_p=last), dict(top_p=tiny), dict(temperature=tiny),
               dict(temperature=np.float32(3.4e38), top_k=8999), dict(top_k=9000), dict(top_k=9001), dict(top_k=512),
               dict(top_k=513), dict(top_p=last, min_p=tiny, top_k=8000), dict(temperature=tiny, min_p=0.5)):
        for u in (0.0, tiny, last):
            check(l, u=u, what=(kw, u), **kw)
    small = (l * np.float32(1e-44)).astype(np.float32)  # subnormal logits, most of them equal
    for kw in (dict(), dict(top_p=0.3), dict(temperature=1e-44, top_p=0.9), dict(temperature=1e-44, top_k=30)):
        check(small, what=kw, **kw)


def test_logits_past_32_bits():
    """Rows that lie more than 2^31 values apart."""
    n, ld = 5003, 2 ** 31 + 3
    buf = torch.empty(ld + n, device="cuda")
    l = logits_of(2, n, 53)
    view = buf.as_strided((2, n), (ld, 1))
    view.copy_(torch.from_numpy(l))
    u = torch.tensor([0.3, 0.9], device="cuda")
    p = torch.full((2,), 0.95, device="cuda")
    idx, prob = q8.sample(view, u, top_p=p)
    torch.cuda.synchronize()
    for r in range(2):
        want, pr = sample_reference.draw(l[r], 1.0, 0, p[r].item(), 0.0, u[r].item())
        assert int(idx[r]) == want and abs(float(prob[r]) - pr) <= 2.0 ** -24 * pr + 2.0 ** -44 * (n * pr + 1)


@pytest.mark.parametrize("rows,n", [(65536, 5), (4097, 65)])
def test_the_most_rows(rows, n):
    rng = np.random.default_rng(59)
    check(logits_of(rows, n, 61), temperature=rng.choice([0.0, 0.7, 1.5], rows), top_k=rng.choice([0, 1, 3], rows),
          top_p=rng.choice([0.5, 1.0], rows), min_p=rng.choice([0.0, 0.2], rows))
