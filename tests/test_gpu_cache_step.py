"""A decode loop with its cache, made of the library's calls: the q, k and v projection,
the cache written, the attention, the output projection; a prompt first, then single
tokens of sequences of different lengths, eager and replayed from a graph."""
import numpy as np
import pytest
import torch

import cache_reference as ref
import oracle
import q8_projection_amd as q8
import synth
from helpers import gate, say

pytestmark = pytest.mark.gpu

STEPS, PAGE, ENTRIES = 5, 32, 4


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """The weights and buffers of one attention layer of `n` sequences that decode together."""

    def __init__(self, bits, heads, kv_heads, dim, k, prompts):
        self.heads, self.kv_heads, self.dim, self.k, self.prompts = heads, kv_heads, dim, k, prompts
        self.bits, n = bits, len(prompts)
        self.wide = (heads + 2 * kv_heads) * dim
        self.w_in = _dev(oracle.quantize_weights(synth.weights(self.wide, k, seed=41)).reshape(self.wide, k // 32 * 34))
        self.w_out = _dev(oracle.quantize_weights(synth.weights(k, heads * dim, seed=42)).reshape(k, heads * dim // 32 * 34))
        self.cache = q8.KVCache(bits, kv_heads, dim, PAGE, n * ENTRIES)
        self.cache.data.random_(0, 256)
        self.table = torch.randperm(n * ENTRIES, device="cuda").to(torch.int32).view(n, ENTRIES)
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.batch = q8.CacheBatch(self.cache, self.table, self.lens)
        self.work = q8.attention_workspace(self.cache, self.batch, heads)
        self.x = torch.empty((n, k), device="cuda")
        self.fused = torch.empty((n, self.wide), device="cuda")
        self.out = torch.empty((n, heads, dim), device="cuda")
        self.lse = torch.empty((n, heads), device="cuda")
        self.y = torch.empty((n, k), device="cuda")

    def split(self, fused):
        a, b = self.heads * self.dim, (self.heads + self.kv_heads) * self.dim
        return (fused[:, :a].unflatten(1, (-1, self.dim)), fused[:, a:b].unflatten(1, (-1, self.dim)),
                fused[:, b:].unflatten(1, (-1, self.dim)))

    def prefill(self, x):
        """The prompts' rows, one after the other."""
        self.lens.copy_(_dev(np.array(self.prompts, np.int32)))
        rows = sum(self.prompts)
        starts = _dev(np.concatenate([[0], np.cumsum(self.prompts)]).astype(np.int32))
        batch = q8.CacheBatch(self.cache, self.table, self.lens, starts, rows, max(self.prompts))
        fused = q8.matmul_rows("f32", self.w_in, self.wide, self.k, x=x)
        q, k, v = self.split(fused)
        q8.cache_append(self.cache, batch, k, v)
        out, _ = q8.attention(self.cache, batch, q)
        return fused, out

    def step(self):
        self.lens.add_(1)
        q8.matmul_rows("f32", self.w_in, self.wide, self.k, x=self.x, out=self.fused)
        q, k, v = self.split(self.fused)
        q8.cache_append(self.cache, self.batch, k, v)
        q8.attention(self.cache, self.batch, q, out=self.out, lse=self.lse, workspace=self.work)
        q8.matmul_rows("f32", self.w_out, self.k, self.heads * self.dim, x=self.out.view(len(self.prompts), -1), residual=self.x, out=self.y)

    def run(self, step, xs, look=None):
        """Prompt and steps; every step's input is the output before it."""
        first = self.prefill(xs)
        last = np.cumsum(self.prompts) - 1
        self.x.copy_(xs[last])
        got = []
        for s in range(STEPS):
            step()
            torch.cuda.synchronize()
            if look:
                look(s, first)
            got.append([t.clone() for t in (self.fused, self.out, self.lse, self.y, self.lens)])
            self.x.copy_(self.y)
        return got


@pytest.mark.parametrize("bits,heads,kv_heads,dim", [(4, 8, 2, 64), (8, 4, 4, 128), (4, 6, 1, 128)])
def test_decode_loop(bits, heads, kv_heads, dim):
    say("decode loop with its cache", bits, heads, kv_heads, dim)
    prompts = [33, 1, 62, 90, 31]
    layer = Layer(bits, heads, kv_heads, dim, 256, prompts)
    xs = _dev(synth.normal(43, (sum(prompts), 256)).astype(np.float32))
    keys = [[] for _ in prompts]  # what the projections gave, kept beside the cache
    values = [[] for _ in prompts]

    def attend(q, s, at, got):
        k, v = ref.values(bits, np.concatenate(keys[s])), ref.values(bits, np.concatenate(values[s]))
        want, _, bound, _, _ = ref.attend(q.astype(np.float64), k, v, at, 1 / np.sqrt(dim))
        assert (np.abs(got - want) <= bound).all(), (s, at)

    def look(step, first):
        starts = np.concatenate([[0], np.cumsum(prompts)])
        if step == 0:
            q, k, v = (t.cpu().numpy() for t in layer.split(first[0]))
            for s in range(len(prompts)):
                r = slice(starts[s], starts[s + 1])
                keys[s], values[s] = [k[r]], [v[r]]
                attend(q[r], s, np.arange(prompts[s]), first[1][r].cpu().numpy())
        q, k, v = (t.cpu().numpy() for t in layer.split(layer.fused))
        for s in range(len(prompts)):
            keys[s].append(k[s:s + 1])
            values[s].append(v[s:s + 1])
            attend(q[s:s + 1], s, np.array([prompts[s] + step]), layer.out[s:s + 1].cpu().numpy())
        r, a = oracle.project("f32", layer.w_out.cpu().numpy(), 256, heads * dim, len(prompts),
                              x=layer.out.view(len(prompts), -1).cpu().numpy(), residual=layer.x.cpu().numpy())
        gate(layer.y.cpu().numpy(), r, a, f"step {step}")

    want = layer.run(layer.step, xs, look)
    graph = torch.cuda.CUDAGraph()
    layer.lens.copy_(_dev(np.array(prompts, np.int32)))
    with torch.cuda.graph(graph):
        layer.step()
    for _ in range(3):
        got = layer.run(graph.replay, xs)
        again = layer.run(layer.step, xs)  # the program's own work between replays
        for w, g, e in zip(want, got, again):
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w, g, e))
