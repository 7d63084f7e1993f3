"""Experts with more tokens than one pass of the kernels takes.

The kernels are chosen by the mean number of tokens an expert gets (vector
instructions up to two, three in the f32 mode), the passes by each expert's own: four
tokens a pass on vector instructions, 8 to 32 on the matrix cores.  The choices here
are few in the mean and many for some experts, so that the vector kernels take
several passes, with every remainder, and then the same choices in a layer whose mean
sends them to the matrix cores.  The tolerances are those of test_gpu_moe.py.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import q8_projection_amd as q8
from helpers import gate, say
from test_gpu_moe import GATE_TOL, _dev, inputs, make

pytestmark = pytest.mark.gpu


def skewed(rows, experts, top_k, counts, seed):
    """Choices [rows][top_k]: expert e of `counts` {e: n} has n tokens spread over the rows, -1 elsewhere."""
    rng = np.random.default_rng(seed)
    ids = np.full((rows, top_k), -1, np.int32)
    for e, n in counts.items():
        free = np.flatnonzero((ids == -1).any(axis=1))
        assert len(free) >= n and e < experts
        for t in rng.permutation(free)[:n]:
            ids[t, rng.choice(np.flatnonzero(ids[t] == -1))] = e
    return ids


# mean at most two (rows * top_k against experts): the vector kernels.  Passes of 4 with
# remainders 0 .. 3, whole and part slices of rows, k longer than what is staged at a
# time (64 blocks in the f32 mode, 128 in the others), ff with a part step and long
VECTOR = [(64, 64, 2, 320, 192, {3: 64, 40: 5, 41: 6, 42: 9, 63: 17, 0: 1, 7: 2}),
          (61, 64, 2, 192, 320, {63: 61, 0: 7, 5: 3, 33: 8, 34: 10}),
          (13, 16, 2, 4160, 64, {15: 13, 2: 5, 3: 6}),
          (13, 16, 2, 64, 4160, {1: 13, 9: 7, 10: 4}),
          (16, 8, 1, 8256, 128, {4: 11, 6: 5}),
          (7, 8, 2, 256, 64, {0: 7, 7: 5, 3: 1}),
          (5, 4, 1, 128, 128, {2: 5}),
          (64, 512, 16, 64, 64, {511: 64, 100: 33, 0: 21, 257: 6}),
          (100, 64, 2, 128, 192, {9: 100, 50: 40, 51: 21})]


def run(mode, rows, experts, top_k, k, ff, ids):
    layer, (wg, wu, wd), _ = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 2100 + rows)
    gates = np.random.default_rng(rows).random((rows, top_k)).astype(np.float32) + np.float32(0.1)
    args = (layer, _dev(x), _dev(ids), _dev(gates), _dev(res))
    y, again = q8.moe_experts(*args), q8.moe_experts(*args)
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, ids, gates, res)
    gate(y.cpu().numpy(), r, a, f"{mode} {rows} rows, {experts} experts, {k} x {ff}")


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows,experts,top_k,k,ff,counts", VECTOR)
def test_several_passes_on_vector_instructions(mode, rows, experts, top_k, k, ff, counts):
    say("passes, vector", mode, rows, experts, top_k, k, ff)
    assert rows % 64 * top_k <= 2 * experts and min(rows, 64) * top_k <= 2 * experts
    run(mode, rows, experts, top_k, k, ff, skewed(rows, experts, top_k, counts, rows + k))


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("n", list(range(1, 20)) + [31, 32, 33, 63, 64])
def test_every_number_of_tokens_on_one_expert(mode, n):
    """n tokens on one expert and a token on another, among 64 rows (vector instructions),
    and the n tokens alone in a layer of one expert (matrix cores from three or four on)."""
    say("tokens", mode, n)
    run(mode, 64, 32, 1, 128, 192, skewed(64, 32, 1, {17: n} if n == 64 else {17: n, 30: 1}, n))
    run(mode, n, 1, 1, 128, 192, np.zeros((n, 1), np.int32))


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows", [6, 13, 61, 64])
def test_a_router_that_prefers_one_expert(mode, rows):
    """The whole layer: every token's first choice is the same expert."""
    experts, top_k, k, ff = 64, 2, 256, 192
    say("hot expert, routed", mode, rows)
    made, (wg, wu, wd), router = make(mode, experts, top_k, k, ff)
    router = router.copy()
    router[:, 0] = 0
    router[37, 0] = 4
    layer = q8.MoeLayer(mode, _dev(wg), _dev(wu), _dev(wd), k, ff, top_k, router=_dev(router))
    x, res = inputs(rows, k, 2500 + rows)
    x[:, 0] = 8
    y, ids, gates = q8.moe(layer, _dev(x), residual=_dev(res))
    torch.cuda.synchronize()
    want_ids, want_gates = ref.route(x, router, top_k)
    assert (want_ids[:, 0] == 37).all() and np.array_equal(ids.cpu().numpy(), want_ids)
    got = gates.cpu().numpy()
    assert (np.abs(got - want_gates) <= GATE_TOL * want_gates).all()
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, want_ids, got, res)
    gate(y.cpu().numpy(), r, a, f"{mode} {rows} rows, one hot expert")
