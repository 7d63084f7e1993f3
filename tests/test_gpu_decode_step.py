"""A decode step made of the library's calls: expert layer, LM head, draw.

Every step is checked in its parts: the expert layer against the 64-bit reference at
the projection's gate, the drawn token against the sampler's definition on the logits
that the GPU computed, and the whole loop replayed from a graph against the eager one.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import oracle
import q8_projection_amd as q8
import sample_reference
import synth
from helpers import gate, say
from test_gpu_moe import _dev, make

pytestmark = pytest.mark.gpu

K, FF, EXPERTS, TOP_K, VOCAB, STEPS = 256, 128, 8, 2, 1003, 3


class Loop:
    """The buffers of a decode loop, and one step on them."""

    def __init__(self, mode, rows):
        self.mode, self.rows = mode, rows
        self.layer, self.blocks, self.router = make(mode, EXPERTS, TOP_K, K, FF)
        head = synth.weights(VOCAB, K, seed=91)
        self.head = _dev(oracle.quantize_weights(head).reshape(VOCAB, K // 32 * 34))
        self.table = _dev(synth.normal(92, (VOCAB, K)).astype(np.float32))
        rng = np.random.default_rng(rows)
        r = np.arange(rows)
        self.par = {"temperature": np.where(r % 4 == 3, 0.0, 0.5 + rng.random(rows)).astype(np.float32),
                    "top_k": np.where(r % 2 == 0, 40, 0).astype(np.int32),
                    "top_p": np.where(r % 3 == 0, 0.9, 1.0).astype(np.float32),
                    "min_p": np.where(r % 5 == 4, 0.02, 0.0).astype(np.float32)}
        self.dev = {k: _dev(v) for k, v in self.par.items()}
        self.u_all = rng.random((STEPS, rows)).astype(np.float32)
        self.u = torch.empty(rows, device="cuda")
        self.start = _dev(synth.normal(93, (rows, K)).astype(np.float32))
        self.x = self.start.clone()
        self.y = torch.empty((rows, K), device="cuda")
        self.logits = torch.empty((rows, VOCAB), device="cuda")
        self.ids = torch.empty((rows, TOP_K), dtype=torch.int32, device="cuda")
        self.gates = torch.empty((rows, TOP_K), device="cuda")
        self.idx = torch.empty(rows, dtype=torch.int32, device="cuda")
        self.prob = torch.empty(rows, device="cuda")
        self.work = self.layer.workspace(rows)
        self.scratch = torch.empty(q8.sample_workspace_bytes(rows, VOCAB), dtype=torch.uint8, device="cuda")

    def step(self):
        q8.moe(self.layer, self.x, residual=self.x, out=self.y, ids=self.ids, gates=self.gates, workspace=self.work)
        if self.rows == 1:
            q8.matvec("f32", self.head, VOCAB, K, x=self.y, out=self.logits.view(-1))
        else:
            q8.matmul_rows("f32", self.head, VOCAB, K, x=self.y, out=self.logits)
        q8.sample(self.logits, self.u, **self.dev, idx=self.idx, prob=self.prob, workspace=self.scratch)
        torch.index_select(self.table, 0, self.idx, out=self.x)

    def run(self, step, look=None):
        self.x.copy_(self.start)
        out = []
        for s in range(STEPS):
            self.u.copy_(_dev(self.u_all[s]))
            before = self.x.clone()
            step()
            torch.cuda.synchronize()
            if look:
                look(s, before)
            out.append([t.clone() for t in (self.y, self.ids, self.gates, self.logits, self.idx, self.prob)])
        return out

    def check(self, s, before):
        x = before.cpu().numpy()
        ids, gates = self.ids.cpu().numpy(), self.gates.cpu().numpy()
        assert np.array_equal(ids, ref.route(x, self.router, TOP_K)[0])
        r, a = ref.experts(self.mode, *self.blocks, K, FF, x, ids, gates, x)
        gate(self.y.cpu().numpy(), r, a, f"step {s}")
        logits = self.logits.cpu().numpy()
        r, a = oracle.project("f32", self.head.cpu().numpy(), VOCAB, K, self.rows, x=self.y.cpu().numpy())
        gate(logits, r, a, f"step {s}, head")
        for row in range(self.rows):
            want, p = sample_reference.draw(logits[row], u=float(self.u_all[s][row]),
                                            **{k: v[row].item() for k, v in self.par.items()})
            assert int(self.idx[row]) == want
            # one f32 rounding, and a unit of 2^-44 for each weight (as in test_gpu_sample.py)
            assert abs(float(self.prob[row]) - p) <= 2.0 ** -24 * p + 2.0 ** -44 * (VOCAB * p + 1)


@pytest.mark.parametrize("mode,rows", [("i8x2", 1), ("i8x2", 6), ("i8", 33), ("f32", 3), ("i8x2", 64)])
def test_decode_loop(mode, rows):
    say("decode loop", mode, rows)
    loop = Loop(mode, rows)
    want = loop.run(loop.step, loop.check)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for _ in range(3):
        got = loop.run(graph.replay)
        again = loop.run(loop.step)  # the program's own work between replays
        for w, g, e in zip(want, got, again):
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w, g, e))
