"""The mixture-of-experts layer where its kernels change their ways: long rows that
are staged in parts, many rows of output, the step from vector to matrix
instructions, tokens spread unevenly over the experts, and streams.  The
tolerances are those of test_gpu_moe.py.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import q8_projection_amd as q8
from helpers import gate, say
from test_gpu_moe import GATE_TOL, _dev, inputs, make

pytestmark = pytest.mark.gpu


def check(mode, rows, experts, top_k, k, ff, renormalize=True):
    say("moe", mode, rows, experts, top_k, k, ff, renormalize)
    layer, (wg, wu, wd), router = make(mode, experts, top_k, k, ff, renormalize)
    x, res = inputs(rows, k, 1300 + rows)
    y, ids, gates = q8.moe(layer, _dev(x), residual=_dev(res))
    torch.cuda.synchronize()
    want_ids, want_gates = ref.route(x, router, top_k, renormalize)
    got = gates.cpu().numpy()
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(got - want_gates) <= GATE_TOL * want_gates).all()
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, want_ids, got, res)
    gate(y.cpu().numpy(), r, a, f"{mode} {rows}x{k}, ff {ff}, {experts} experts")


# one token, a few, and more than four an expert; k and ff longer than what is staged
# at a time, with a part block of a step; so many columns that no tile is shared
@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows,experts,top_k,k,ff", [(1, 2, 1, 8256, 64), (3, 2, 1, 8256, 64), (20, 2, 2, 8256, 128),
                                                     (40, 2, 1, 4160, 192), (2, 3, 2, 64, 8256), (64, 2, 2, 64, 4160),
                                                     (33, 1, 1, 16448, 64)])
def test_long_rows_and_columns(mode, rows, experts, top_k, k, ff):
    check(mode, rows, experts, top_k, k, ff)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows,experts,top_k", [(4, 2, 1), (6, 2, 1), (7, 2, 1), (5, 2, 1), (8, 2, 1), (9, 2, 1), (3, 3, 2), (4, 3, 2), (6, 3, 2), (7, 3, 2), (10, 3, 2), (26, 3, 1), (64, 8, 1)])
def test_number_of_tokens_an_expert(mode, rows, experts, top_k):
    check(mode, rows, experts, top_k, 320, 192)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
@pytest.mark.parametrize("rows", [1, 4, 24])
def test_gates_over_all_experts(mode, rows):
    check(mode, rows, 7, 2, 192, 128, renormalize=False)


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_tokens_spread_unevenly(mode):
    """64 tokens on one expert, one and a few on others, none on the rest."""
    rows, experts, top_k, k, ff = 64, 8, 3, 320, 192
    layer, (wg, wu, wd), _ = make(mode, experts, top_k, k, ff)
    x, res = inputs(rows, k, 1401)
    rng = np.random.default_rng(11)
    ids = np.full((rows, top_k), -1, np.int32)
    ids[:, 0] = 3
    ids[40, 1] = 0
    ids[5:22, 2] = 7
    ids[9:18, 1] = 4
    gates = rng.random((rows, top_k)).astype(np.float32)
    y = q8.moe_experts(layer, _dev(x), _dev(ids), _dev(gates), residual=_dev(res))
    torch.cuda.synchronize()
    r, a = ref.experts(mode, wg, wu, wd, k, ff, x, ids, gates, res)
    gate(y.cpu().numpy(), r, a, f"uneven {mode}")


@pytest.mark.parametrize("mode", ["f32", "i8", "i8x2"])
def test_a_token_that_is_no_number_stays_alone(mode):
    rows, experts, top_k, k, ff = 40, 4, 2, 256, 128
    layer, _, _ = make(mode, experts, top_k, k, ff)
    x, _ = inputs(rows, k, 1501)
    ids = _dev(np.random.default_rng(5).permuted(np.tile(np.arange(experts, dtype=np.int32), (rows, 1)), axis=1)[:, :top_k].copy())
    gates = torch.full((rows, top_k), 0.5, device="cuda")
    want = q8.moe_experts(layer, _dev(x), ids, gates)
    x[7, 100] = np.nan
    x[23, 5] = np.inf
    got = q8.moe_experts(layer, _dev(x), ids, gates)
    torch.cuda.synchronize()
    others = [i for i in range(rows) if i not in (7, 23)]
    assert torch.equal(want[others], got[others]) and torch.isfinite(got[others]).all()


def test_counters_are_zero_after_a_call_that_uses_them_all():
    layer, _, _ = make("i8x2", 16, 4, 512, 256)
    work = layer.workspace(64)
    for rows in (64, 61, 3):
        q8.moe(layer, _dev(inputs(rows, 512, 1600)[0]), workspace=work)
        torch.cuda.synchronize()
        assert not work[:(32 * 32 + 512) * 4].any()


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_stream_orders_what_the_call_allocates(raw):
    """The workspace that a call makes for itself is cleared on the call's stream, not on
    a busy current one, and is not memory that the current one still uses."""
    rows, k = 24, 256
    layer, _, _ = make("i8x2", 8, 2, k, 128)
    x = _dev(inputs(rows, k, 1700)[0])
    want = q8.moe(layer, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = torch.full((layer.workspace_bytes(rows),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(100_000_000)
    got = q8.moe(layer, x, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
