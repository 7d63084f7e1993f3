"""The sampler on the GPU against its definition.

Indices are equal.  A probability is one f32 rounding (2^-24 relative) of a
quotient of integer weights; each weight may be one unit (2^-44 of the largest)
off where the device's f64 exp and the host's differ in the last bit, so the
kept sum by n units and the weight by one: 2^-24 + 2^-44 (n + 1 / prob) relative.
"""
import math

import numpy as np
import pytest
import torch

import q8_projection_amd as q8
import sample_reference as ref
from helpers import say

pytestmark = pytest.mark.gpu


def check(logits, temperature=None, top_k=None, top_p=None, min_p=None, u=None, pad=0, what="", **kw):
    """Draw on the GPU from numpy inputs and compare every row."""
    rows, n = logits.shape
    buf = torch.full((rows, n + pad), 9e9, device="cuda")
    buf[:, :n] = torch.from_numpy(np.ascontiguousarray(logits, dtype=np.float32)).cuda()
    u = np.random.default_rng(rows + n).random(rows) if u is None else u
    par = {}
    for name, v, dtype in (("temperature", temperature, np.float32), ("top_k", top_k, np.int32),
                           ("top_p", top_p, np.float32), ("min_p", min_p, np.float32), ("u", u, np.float32)):
        par[name] = None if v is None else np.broadcast_to(np.asarray(v, dtype), (rows,)).copy()
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in par.items()}
    idx, prob = q8.sample(buf[:, :n], **dev, **kw)
    torch.cuda.synchronize()
    idx, prob = idx.cpu().numpy(), prob.cpu().numpy()
    off = {"temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0}
    for r in range(rows):
        args = {k: (off[k] if v is None else v[r].item()) for k, v in par.items()}
        want, p = ref.draw(logits[r], **args)
        assert idx[r] == want, (what, r, args, int(idx[r]), want)
        tol = 2.0 ** -24 * p + 2.0 ** -44 * (n * p + 1)
        assert abs(float(prob[r]) - p) <= tol, (what, r, args, float(prob[r]), p)
    return idx, prob


def logits_of(rows, n, seed, spread=2.5):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(rows, n)) * spread
    lead = rng.integers(0, n, (rows, 8))
    np.put_along_axis(l, lead, np.take_along_axis(l, lead, 1) + 3 * spread * rng.random((rows, 8)), 1)
    return l.astype(np.float32)


KINDS = {"plain": {}, "temperature": dict(temperature=0.7), "topk": dict(temperature=0.9, top_k=40), "k1": dict(top_k=1),
         "topp": dict(temperature=1.1, top_p=0.9), "both": dict(temperature=0.8, top_k=50, top_p=0.95),
         "minp": dict(temperature=1.3, min_p=0.05), "all": dict(temperature=1.2, top_k=200, top_p=0.97, min_p=0.001),
         "wide": dict(temperature=1.5, top_k=3000, top_p=0.999)}


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,n,pad", [(3, 1, 0), (5, 2, 1), (4, 63, 0), (4, 64, 3), (4, 65, 0), (9, 1000, 1),
                                        (3, 4097, 0), (2, 32003, 5), (1, 151936, 0), (70, 5000, 2)])
def test_draws(kind, rows, n, pad):
    say("sample", kind, rows, n, pad)
    check(logits_of(rows, n, 17 * n + rows), pad=pad, what=(kind, n), **KINDS[kind])


@pytest.mark.parametrize("spread", [0.0001, 0.05, 1.0, 8.0])
def test_flat_and_peaked_rows(spread):
    """From nearly equal logits (many tokens in one bin of the histogram) to peaked ones."""
    say("spread", spread)
    l = logits_of(6, 30011, 5, spread)
    for kw in (dict(), dict(top_p=0.5), dict(top_k=5000), dict(top_k=20000, top_p=0.9), dict(top_p=0.999, min_p=1e-4),
               dict(temperature=100.0, top_p=0.7), dict(temperature=1e6, top_k=9000), dict(temperature=1e-4, top_p=0.9)):
        check(l, what=(spread, kw), **kw)


def test_ties_go_to_the_lowest_index():
    l = np.zeros((8, 10000), np.float32)
    l[:, 1::2] = -0.0
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.9999, 1.0, -1.0, float("nan")], np.float32)
    idx, prob = check(l, u=u)
    assert idx[0] == 0 and idx[1] == 2500 and idx[5] == 9999 and idx[6] == 0 and idx[7] == 9999
    idx, prob = check(l, u=u, top_p=0.5)
    assert idx[5] == 4999 and prob[0] == np.float32(1 / 5000)
    check(l, u=u, top_k=7777)
    check(l, u=u, top_k=9000, top_p=0.125)
    check(l, u=u, temperature=0.0)
    # a tied bulk below and above other tokens
    l[:, 300:310] = 1.5
    l[:, 400:900] = -2.0
    for kw in (dict(), dict(top_k=9600), dict(top_p=0.9), dict(top_k=5, top_p=0.3), dict(min_p=0.2), dict(min_p=1.0),
               dict(min_p=2.0)):
        check(l, u=u, what=kw, **kw)


def test_masked_rows_infinities_and_nan():
    low, inf, nan = np.finfo(np.float32).min, np.inf, np.nan
    l = logits_of(10, 3001, 11)
    l[0] = -inf
    l[1] = nan
    l[2] = low                        # every token masked with the type's lowest value: all equal
    l[3, :-1] = -inf                  # one candidate
    l[4, ::2] = low
    l[5, 1::3] = nan
    l[6, 7] = inf
    l[7, [5, 9, 2000]] = inf          # several: equal weights among them
    l[8, :] = -inf
    l[8, [3, 2999]] = low
    l[9, 100:] = -inf
    for kw in (dict(), dict(top_k=50), dict(top_p=0.9), dict(temperature=0.0), dict(temperature=float("inf")),
               dict(temperature=float("nan")), dict(temperature=-1.0), dict(top_k=20, top_p=0.5, min_p=0.1),
               dict(top_k=2 ** 31 - 1), dict(top_k=-5), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=float("nan")),
               dict(min_p=float("nan")), dict(temperature=1e-38), dict(temperature=3e38)):
        for u in (0.0, 0.6, 0.99999994):
            check(l, u=u, what=(kw, u), **kw)


def test_mixed_rows_share_a_call():
    rows, n = 64, 20011
    rng = np.random.default_rng(2)
    check(logits_of(rows, n, 3), temperature=rng.choice([0.0, 0.5, 1.0, 1.7], rows), top_k=rng.choice([0, 1, 30, 600, 5000], rows),
          top_p=rng.choice([0.5, 0.9, 1.0], rows), min_p=rng.choice([0.0, 0.02, 0.3], rows), pad=13)


def test_same_call_same_draw_workspace_streams_and_replays():
    rows, n = 6, 50257
    a = [torch.from_numpy(logits_of(rows, n, 40 + i)).cuda() for i in range(3)]
    small = torch.from_numpy(logits_of(2, 700, 50)).cuda()
    u, u2 = torch.rand(rows, device="cuda"), torch.rand(2, device="cuda")
    kw = dict(temperature=torch.full((rows,), 0.9, device="cuda"), top_p=torch.tensor([0.9, 1.0] * 3, device="cuda"),
              top_k=torch.tensor([0, 0, 40, 2000, 0, 64], dtype=torch.int32, device="cuda"))
    want = [q8.sample(l, u, **kw) for l in a]
    want_small = q8.sample(small, u2)
    work = torch.zeros(q8.sample_workspace_bytes(rows, n), dtype=torch.uint8, device="cuda")
    idx, prob = torch.full((rows + 3,), -7, dtype=torch.int32, device="cuda"), torch.full((rows + 3,), -7.0, device="cuda")
    x = a[0].clone()
    side = torch.cuda.Stream()
    q8.sample(x, u, **kw, workspace=work, idx=idx[:rows], prob=prob[:rows])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.sample(x, u, **kw, workspace=work, idx=idx[:rows], prob=prob[:rows])
    for _ in range(3):
        for l, w in zip(a, want):
            x.copy_(l)
            graph.replay()
            got_small = q8.sample(small, u2, workspace=work)
            torch.cuda.synchronize()
            assert torch.equal(idx[:rows], w[0]) and torch.equal(prob[:rows], w[1])
            assert torch.equal(got_small[0], want_small[0]) and torch.equal(got_small[1], want_small[1])
            eager = q8.sample(l, u, **kw, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(eager[0], w[0]) and torch.equal(eager[1], w[1])
    assert (idx[rows:] == -7).all() and (prob[rows:] == -7).all()


def test_empty_and_refused():
    e = q8.sample(torch.empty((0, 10), device="cuda"), torch.empty(0, device="cuda"))
    assert e[0].numel() == 0 and e[1].numel() == 0
    l, u = torch.zeros((2, 10), device="cuda"), torch.zeros(2, device="cuda")
    for bad in (l.double(), l.t(), l.cpu(), l[0], torch.zeros((2, 20), device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            q8.sample(bad, u)
    with pytest.raises(ValueError):
        q8.sample(l, u, top_k=torch.zeros(2, device="cuda"))
    with pytest.raises(q8.Q8Error, match="Q8_E_SHAPE"):
        q8.sample(l[:1].expand(2, 10), u)
    with pytest.raises(q8.Q8Error, match="Q8_E_SHAPE"):
        q8.sample(l, u, workspace=torch.zeros(0, dtype=torch.uint8, device="cuda").new_zeros(16))


def test_more_rows_than_one_pass_takes():
    rows, n = 2100, 300
    rng = np.random.default_rng(8)
    check(logits_of(rows, n, 9), temperature=rng.choice([0.0, 0.8, 1.5], rows), top_k=rng.choice([0, 4, 290], rows),
          top_p=rng.choice([0.3, 1.0], rows))


@pytest.mark.parametrize("rows,n", [(1, 262144), (2, 524287), (20, 70001)])
def test_long_rows(rows, n):
    say("long rows", rows, n)
    l = logits_of(rows, n, n)
    for kw in (dict(), dict(top_p=0.95), dict(top_k=1500, top_p=0.9), dict(top_k=100), dict(temperature=2.0, min_p=0.01)):
        check(l, what=kw, **kw)


@pytest.mark.parametrize("kind", ["plain", "topp", "all", "minp", "wide"])
@pytest.mark.parametrize("rows,n", [(40, 30011), (130, 9001), (256, 4100)])
def test_rows_that_share_the_card(kind, rows, n):
    """As many workgroups a row as the number of rows leaves."""
    say("sample", kind, rows, n)
    check(logits_of(rows, n, 77 + rows), what=kind, **KINDS[kind])
