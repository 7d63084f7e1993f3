"""The mixture-of-experts layer on the GPU against the 64-bit reference.

Outputs are held to the projection's gate (helpers.py): |y - Y| <= 1e-5 |Y| +
2^-40 A and one f32 step where the second term is small.  Gates are one f32
rounding of a f64 quotient: 2^-24 relative, and 2^-40 for the f64 arithmetic
before it (at most 512 terms of 2^-52).
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import oracle
import q8_projection_amd as q8
import synth
from helpers import gate, say

pytestmark = pytest.mark.gpu

GATE_TOL = 2.0 ** -24 + 2.0 ** -40


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


_layers = {}


def make(mode, experts, top_k, k, ff, renormalize=True):
    """(layer, numpy blocks, numpy router) of a seeded layer."""
    key = (experts, k, ff)
    if key not in _layers:
        seed = 7000 + experts * 131 + k * 7 + ff
        def mat(i, n, c):
            w = synth.weights(experts * n, c, seed=seed + i)
            return oracle.quantize_weights(w).reshape(experts, n, c // 32 * 34)
        router = (synth.normal(seed + 9, (experts, k)) / np.sqrt(k)).astype(np.float32)
        _layers[key] = (mat(1, ff, k), mat(2, ff, k), mat(3, k, ff), router)
    wg, wu, wd, router = _layers[key]
    layer = q8.MoeLayer(mode, _dev(wg), _dev(wu), _dev(wd), k, ff, top_k, router=_dev(router),
                        renormalize=renormalize)
    return layer, (wg, wu, wd), router


def inputs(rows, k, seed):
    return synth.activations(rows, k, seed=seed).astype(np.float32), synth.normal(seed + 1, (rows, k)).astype(np.float32)


# modes x: one token, small and odd batches, a full slice, more than one slice;
# the smallest sizes, block counts that are no multiple of a step's eight, all
# tokens on one expert, more experts than pairs, the most choices
SHAPES = [(1, 8, 2, 256, 128), (1, 1, 1, 64, 64), (2, 4, 4, 192, 320), (5, 6, 3, 1088, 192), (3, 512, 16, 128, 64),
          (17, 3, 2, 320, 576), (64, 1, 1, 256, 64), (64, 16, 4, 512, 256), (70, 5, 2, 128, 192), (130, 2, 1, 64, 128)]


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows,experts,top_k,k,ff", SHAPES)
def test_layer_against_the_reference(mode, rows, experts, top_k, k, ff):
    say("moe", mode, rows, experts, top_k, k, ff)
    layer, (wg, wu, wd), router = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 300 + rows)
    y, ids, gates = q8.moe(layer, _dev(x), residual=_dev(res))
    torch.cuda.synchronize()
    want_ids, want_gates = ref.route(x, router, top_k)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = gates.cpu().numpy()
    assert (np.abs(got - want_gates) <= GATE_TOL * want_gates).all()
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, want_ids, got, res)
    gate(y.cpu().numpy(), r, a, f"{mode} {rows}x{k}, {experts} experts")


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("rows,experts,top_k,k", [(1, 64, 8, 2048), (9, 100, 6, 1984), (64, 65, 1, 64), (65, 512, 16, 128)])
def test_router(rows, experts, top_k, k, renormalize):
    say("route", rows, experts, top_k, k, renormalize)
    layer, _, router = make("i8x2", experts, top_k, k, 64, renormalize)
    x, _ = inputs(rows, k, 410)
    ids, gates = q8.moe_route(layer, _dev(x))
    torch.cuda.synchronize()
    want_ids, want_gates = ref.route(x, router, top_k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(gates.cpu().numpy() - want_gates) <= GATE_TOL * want_gates).all()


def test_router_ties_go_to_the_lowest_expert():
    experts, k, top_k = 130, 64, 4
    row = synth.normal(5, (1, k)).astype(np.float32)
    router = np.repeat(row, experts, axis=0)
    router[70] *= 2
    wd = np.zeros((experts, 64, k // 32 * 34), np.uint8)
    layer = q8.MoeLayer("i8", _dev(wd), _dev(wd), _dev(wd), k, 64, top_k, router=_dev(router))
    ids, gates = q8.moe_route(layer, _dev(np.concatenate([row, -row, 0 * row])))
    torch.cuda.synchronize()
    assert ids.cpu().tolist() == [[70, 0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 3]]
    assert torch.equal(gates[1:].cpu(), torch.full((2, 4), 0.25))


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_given_choices_padded_repeated_and_out_of_range(mode):
    rows, experts, top_k, k, ff = 11, 6, 3, 256, 192
    layer, (wg, wu, wd), _ = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 520)
    rng = np.random.default_rng(3)
    ids = rng.integers(0, experts, (rows, top_k)).astype(np.int32)
    ids[0] = [2, 2, 5]
    ids[1] = [4, 4, 4]
    ids[2] = [-1, 3, 2 ** 31 - 1]
    ids[3] = [experts, -2 ** 31, 0]
    ids[-3:] = -1
    gates = rng.random((rows, top_k)).astype(np.float32)
    gates[4, 0] = 0.0
    gates[5, 1] = -0.5
    # rows behind the batch stay as they were
    out = torch.full((rows + 4, k), float("nan"), device="cuda")
    y = q8.moe_experts(layer, _dev(x), _dev(ids), _dev(gates), residual=_dev(res), out=out[:rows])
    none = q8.moe_experts(layer, _dev(x), _dev(ids), _dev(gates))
    torch.cuda.synchronize()
    assert torch.isnan(out[rows:]).all()
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, ids, gates, res)
    gate(y.cpu().numpy(), r, a, f"given {mode}")
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, ids, gates)
    gate(none.cpu().numpy(), r, a, f"given {mode}, no residual")
    assert not none[-3:].any() and np.array_equal(y[-3:].cpu().numpy(), res[-3:])


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_layer_is_route_then_experts_bit_for_bit(mode):
    rows, experts, top_k, k, ff = 7, 12, 3, 320, 128
    layer, _, _ = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 630)
    xd, rd = _dev(x), _dev(res)
    y, ids, gates = q8.moe(layer, xd, residual=rd)
    ids2, gates2 = q8.moe_route(layer, xd)
    y2 = q8.moe_experts(layer, xd, ids2, gates2, residual=rd)
    in_place = rd.clone()
    q8.moe(layer, xd, residual=in_place, out=in_place)
    torch.cuda.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(gates, gates2) and torch.equal(y, y2) and torch.equal(y, in_place)


def test_one_expert_is_the_projections_of_the_library():
    """One expert with gate 1 is matmul_rows, the activation between, matmul_rows."""
    rows, k, ff = 4, 512, 256
    layer, (wg, wu, wd), _ = make("i8x2", 1, 1, k, ff)
    x, _ = inputs(rows, k, 710)
    xd = _dev(x)
    y, ids, gates = q8.moe(layer, xd)
    hi, lo, s = q8.quantize_act("i8x2", xd)
    g = q8.matmul_rows("i8x2", _dev(wg[0]), ff, k, hi=hi, lo=lo, scale=s)
    u = q8.matmul_rows("i8x2", _dev(wu[0]), ff, k, hi=hi, lo=lo, scale=s)
    h = (g.double() / (1.0 + torch.exp(-g.double())) * u.double()).float()
    hi, lo, s = q8.quantize_act("i8x2", h)
    want = q8.matmul_rows("i8x2", _dev(wd[0]), k, ff, hi=hi, lo=lo, scale=s)
    torch.cuda.synchronize()
    assert not ids.any() and torch.equal(gates, torch.ones_like(gates))
    # both round the same f64 sum once, added in another order: at most one f32 step
    assert (y - want).abs().max() <= 2.0 ** -23 * want.abs().max()


def test_workspace_serves_layer_after_layer():
    """One zero-filled workspace, calls of different layers, sizes and modes in a row."""
    cases = [("i8x2", 5, 6, 3, 1088, 192), ("f32", 1, 8, 2, 256, 128), ("i8", 17, 3, 2, 320, 576),
             ("i8x2", 1, 8, 2, 256, 128), ("i8x2", 64, 16, 4, 512, 256)]
    made = [(make(m, e, t, k, f)[0], _dev(inputs(r, k, 800 + r)[0])) for m, r, e, t, k, f in cases]
    alone = [q8.moe(layer, x) for layer, x in made]
    work = torch.zeros(max(layer.workspace_bytes(x.shape[0]) for layer, x in made), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for (layer, x), want in zip(made, alone):
            got = q8.moe(layer, x, workspace=work)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert not work[:4096].any()


def test_replayed_graph_and_another_stream():
    rows, experts, top_k, k, ff = 3, 8, 2, 256, 128
    layer, _, _ = make("i8x2", experts, top_k, k, ff)
    xs = [_dev(inputs(rows, k, 900 + i)[0]) for i in range(4)]
    want = [q8.moe(layer, x) for x in xs]
    work, x = layer.workspace(rows), xs[0].clone()
    out, ids = torch.empty((rows, k), device="cuda"), torch.empty((rows, top_k), dtype=torch.int32, device="cuda")
    gates = torch.empty((rows, top_k), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q8.moe(layer, x, out=out, ids=ids, gates=gates, workspace=work)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.moe(layer, x, out=out, ids=ids, gates=gates, workspace=work)
    for _ in range(3):
        for v, w in zip(xs, want):
            x.copy_(v)
            graph.replay()
            eager = q8.moe(layer, v, stream=side)  # the program's own work between replays
            torch.cuda.synchronize()
            assert torch.equal(out, w[0]) and torch.equal(ids, w[1]) and torch.equal(gates, w[2])
            assert torch.equal(eager[0], w[0])


def test_wrapper_refuses_wrong_tensors():
    layer, _, _ = make("i8x2", 8, 2, 256, 128)
    x = torch.zeros((2, 256), device="cuda")
    for bad in (x.double(), x[:, :192], x.t(), torch.zeros((2, 512), device="cuda")[:, ::2], x.cpu()):
        with pytest.raises(ValueError):
            q8.moe(layer, bad)
    with pytest.raises(ValueError):
        q8.moe_experts(layer, x, torch.zeros((2, 2), dtype=torch.int64, device="cuda"), torch.zeros((2, 2), device="cuda"))
    with pytest.raises(q8.Q8Error, match="Q8_E_SHAPE"):
        q8.moe(layer, x, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
