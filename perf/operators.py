"""The measured cases of the decode-step operators: the mixture-of-experts layer
(router, gate, up and down projections of the chosen experts, Q8_0 weights) and
the sampler that draws the next token from the LM head's logits.

A case is a dict of plain values.  `prepare` makes its inputs on the GPU from a
seed, `run` makes one pass (the plain torch form, or the package's entry points
where `own` is true), `exact` computes the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 32
UNIT = float(1 << 44)  # sampling weights are multiples of 2^-44 of the largest


# ------------------------------------------------------------------ the cases

def _moe(name, mode, rows, experts, top_k, k, ff, given=False, residual=False):
    return {"name": name, "op": "experts" if given else "moe", "mode": mode, "rows": rows, "experts": experts,
            "top_k": top_k, "k": k, "ff": ff, "residual": residual}


def _sample(name, rows, n, kind, spread, masked=False, pad=0):
    return {"name": name, "op": "sample", "rows": rows, "n": n, "kind": kind, "spread": spread, "masked": masked,
            "pad": pad}


def listed():
    return [
        # the smallest layer: one token, matrices of the tiny matvec's size; all latency
        _moe("moe_tiny_token", "i8x2", 1, 8, 2, 1024, 256),
        # one decode step of one sequence through many small experts
        _moe("moe_token_small_experts", "i8x2", 1, 64, 8, 2048, 1408, residual=True),
        # one decode step through two large experts (the dense layer's up/gate/down shapes)
        _moe("moe_token_large_experts", "i8x2", 1, 8, 2, 4096, 14336),
        # eight sequences decoding together
        _moe("moe_batch8_small_experts", "i8x2", 8, 64, 8, 2048, 1408),
        # odd sizes, f32 activations with f64 sums
        _moe("moe_f32_odd", "f32", 3, 12, 3, 1984, 1216),
        # sixteen sequences, large experts, one-word activations: the largest
        _moe("moe_batch16_large_experts", "i8", 16, 8, 2, 4096, 14336, residual=True),
        # a chunk of 64 rows through small experts: nearly every expert is read, about 8 rows each
        _moe("moe_rows64_small_experts", "i8x2", 64, 64, 8, 2048, 1408),
        # a router of the caller's own: padded rows (no expert), a repeated choice
        _moe("experts_given_padded13", "i8x2", 13, 24, 4, 2048, 704, given=True, residual=True),
        # the usual serving choice, one sequence: temperature, top-k and top-p over the whole vocabulary
        _sample("sample_one_row", 1, 151936, "topk_topp", 2.5),
        # a batch whose sequences each ask for something else; some tokens masked; rows of a padded logits buffer
        _sample("sample_64_mixed", 64, 151936, "mixed", 2.5, masked=True, pad=64),
        # nucleus sampling without top-k, odd vocabulary
        _sample("sample_topp_odd", 8, 32003, "topp", 3.0),
        # plain temperature sampling of many sequences (min-p on half of them)
        _sample("sample_temperature_256", 256, 50257, "minp", 2.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.4:
        n = _log_int(rng, 1000, 152064)
        return {"op": "sample", "rows": _log_int(rng, 1, 256 if n < 40000 else 64), "n": n,
                "kind": rng.choice(["topk_topp", "mixed", "topp", "minp", "topk"]),
                "spread": round(rng.uniform(0.7, 4.0), 3), "masked": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 1, 64])}
    op = "experts" if rng.random() < 0.3 else "moe"
    experts = _log_int(rng, 4, 128)
    top_k = rng.randint(1, min(8, experts))
    k = 64 * _log_int(rng, 8, 64)
    ff = 64 * _log_int(rng, 2, max(2, min(224, int(8 * 14336 * 4096 / (experts * k * 64)))))
    return {"op": op, "mode": rng.choice(["i8x2", "i8x2", "i8", "f32"]), "rows": _log_int(rng, 1, 64 if k * ff * experts < 1 << 28 else 16),
            "experts": experts, "top_k": top_k, "k": k, "ff": ff, "residual": rng.random() < 0.5}


def work(case):
    if case["op"] == "sample":
        rows, n = case["rows"], case["n"]
        return {"bytes": rows * (4 * n + 28), "flops": 2 * rows * n}
    rows, e, tk, k, ff = (case[x] for x in ("rows", "experts", "top_k", "k", "ff"))
    used = e * (1.0 - (1.0 - tk / e) ** rows)  # distinct experts that `rows` even choices of `top_k` reach
    return {"bytes": int(used * 3 * ff * k * 34 / 32 + rows * k * 4 * (3 if case["residual"] else 2)
                         + rows * tk * 8 + (e * k * 4 if case["op"] == "moe" else 0)),
            "flops": rows * tk * 6 * k * ff + (2 * rows * e * k if case["op"] == "moe" else 0)}


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _q8_blocks(gen, experts, n, k):
    """Q8_0 blocks [experts][n][k/32][34] (uint8) of normal weights of deviation 1/sqrt(k)."""
    out = torch.empty((experts, n, k // BLOCK, 34), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (n * k))  # experts a pass: bounded scratch
    for e0 in range(0, experts, step):
        m = min(step, experts - e0)
        w = torch.randn((m, n, k // BLOCK, BLOCK), device="cuda", generator=gen) / math.sqrt(k)
        d = (w.abs().amax(-1, keepdim=True) / 127.0).half()
        q = (w / d.float()).round_().clamp_(-127, 127).to(torch.int8)
        out[e0:e0 + m, ..., :2] = d.contiguous().view(torch.uint8).view(m, n, k // BLOCK, 2)
        out[e0:e0 + m, ..., 2:] = q.view(torch.uint8)
    return out.view(experts, n, k // BLOCK * 34)


def _params(gen, rows, kind):
    """Per-row sampling parameters as a serving loop holds them, and the random numbers."""
    temperature = 0.6 + 0.8 * torch.rand(rows, device="cuda", generator=gen)
    top_k = torch.zeros(rows, dtype=torch.int32, device="cuda")
    top_p = torch.ones(rows, device="cuda")
    min_p = torch.zeros(rows, device="cuda")
    u = torch.rand(rows, device="cuda", generator=gen)
    r = torch.arange(rows, device="cuda")
    if kind in ("topk_topp", "topk"):
        top_k += torch.randint(20, 101, (rows,), device="cuda", generator=gen, dtype=torch.int32)
    if kind in ("topk_topp", "topp"):
        top_p = 0.8 + 0.19 * torch.rand(rows, device="cuda", generator=gen)
    if kind == "minp":
        min_p = torch.where(r % 2 == 0, 0.05, 0.0).float()
    if kind == "mixed":  # greedy, top-k, top-p, both, min-p, plain, a large top-k, everything
        k = torch.tensor([0, 40, 0, 50, 0, 0, 2000, 64], dtype=torch.int32, device="cuda")
        p = torch.tensor([1.0, 1.0, 0.9, 0.95, 1.0, 1.0, 0.99, 0.9], device="cuda")
        mp = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.1, 0.0, 0.0, 0.02], device="cuda")
        top_k, top_p, min_p = k[r % 8], p[r % 8], mp[r % 8]
        temperature = torch.where(r % 8 == 0, 0.0, temperature)
    return {"temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "u": u}


def _inputs(case, seed):
    gen = _gen(seed)
    rows = case["rows"]
    if case["op"] == "sample":
        n = case["n"]
        buf = torch.randn((rows, n + case["pad"]), device="cuda", generator=gen) * case["spread"]
        logits = buf[:, :n]
        # a language model's head: a few tokens stand out of the bulk
        lead = torch.randint(0, n, (rows, 12), device="cuda", generator=gen)
        logits.scatter_add_(1, lead, 3 * case["spread"] * torch.rand((rows, 12), device="cuda", generator=gen))
        if case["masked"]:  # tokens that a grammar forbids: -inf, or the type's lowest value on every third row
            drop = torch.rand((rows, n), device="cuda", generator=gen) < 0.1
            low = torch.where(torch.arange(rows, device="cuda") % 3 == 0, torch.finfo(torch.float32).min, -math.inf)
            logits.copy_(torch.where(drop, low[:, None], logits))
        return {"logits": logits, **_params(gen, rows, case["kind"])}
    e, tk, k, ff = (case[x] for x in ("experts", "top_k", "k", "ff"))
    x = torch.randn((rows, k), device="cuda", generator=gen)
    x *= torch.where(torch.rand(k, device="cuda", generator=gen) < 0.005, 20.0, 1.0)  # outlier channels
    state = {"x": x, "w_gate": _q8_blocks(gen, e, ff, k), "w_up": _q8_blocks(gen, e, ff, k),
             "w_down": _q8_blocks(gen, e, k, ff),
             "residual": torch.randn((rows, k), device="cuda", generator=gen) if case["residual"] else None}
    if case["op"] == "moe":
        state["router"] = torch.randn((e, k), device="cuda", generator=gen) / math.sqrt(k)
    else:
        ids = torch.rand((rows, e), device="cuda", generator=gen).argsort(1)[:, :tk].to(torch.int32)
        if rows > 1:
            ids[-max(1, rows // 5):] = -1        # rows that pad the batch: no expert
        if tk > 1:
            ids[0, 1] = ids[0, 0]                # the same expert twice
        state["ids"] = ids.contiguous()
        state["gates"] = torch.rand((rows, tk), device="cuda", generator=gen)
    return state


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        import q8_projection_amd as q8
        state["q8"] = q8
        if case["op"] == "sample":
            state["workspace"] = torch.zeros(q8.sample_workspace_bytes(case["rows"], case["n"]), dtype=torch.uint8,
                                             device="cuda")
        else:
            state["layer"] = q8.MoeLayer(case["mode"], state["w_gate"], state["w_up"], state["w_down"], case["k"],
                                         case["ff"], case["top_k"], router=state.get("router"))
            state["workspace"] = state["layer"].workspace(case["rows"])
    return state


# ------------------------------------------------------------- the plain form

def _dequant(blocks, k):
    """f64 weights [n][k] of one expert's Q8_0 blocks [n][k/32*34]."""
    b = blocks.view(blocks.shape[0], k // BLOCK, 34)
    d = b[..., :2].contiguous().view(torch.float16).double()
    return (b[..., 2:].contiguous().view(torch.int8).double() * d).view(blocks.shape[0], k)


def _half_away(v):
    return torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v))


def _act(mode, x):
    """f64 values that the activation's int8 words and block scales stand for (f32 mode: x)."""
    if mode == "f32":
        return x.double()
    b = x.view(x.shape[0], -1, BLOCK)
    # f32 quotients, correctly rounded (a f64 quotient of f32 values, rounded once more, is); the
    # rounding half away is exact in f64
    s = (b.abs().amax(-1, keepdim=True).double() / 127.0).float().double()
    one = torch.where(s == 0, torch.ones_like(s), s)
    hi = _half_away((b.double() / one).float().double()).clamp(-127, 127)
    v = hi
    if mode == "i8x2":
        rest = (b.double() - s * hi).float().double()  # exact product and difference, rounded once
        v = hi + _half_away((rest * 128.0 / one).float().double()).clamp(-127, 127) / 128.0
    return torch.where(s == 0, torch.zeros_like(v), v * s).view(x.shape[0], -1)


def _run_route(state, case):
    z = (state["x"].double() @ state["router"].double().t()).float()
    order = torch.sort(z, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :case["top_k"]], order.values[:, :case["top_k"]]
    p = torch.exp(top.double() - z.amax(1, keepdim=True).double())
    return ids.to(torch.int32), (p / p.sum(1, keepdim=True)).float()


def _run_experts(state, case, ids, gates):
    mode, k, ff, e = case["mode"], case["k"], case["ff"], case["experts"]
    a = _act(mode, state["x"])
    y = torch.zeros_like(state["x"], dtype=torch.float64) if state["residual"] is None else state["residual"].double()
    for i in torch.unique(ids[(ids >= 0) & (ids < e)]).tolist():
        t, slot = torch.nonzero(ids == i, as_tuple=True)
        g = (a[t] @ _dequant(state["w_gate"][i], k).t()).float().double()
        up = (a[t] @ _dequant(state["w_up"][i], k).t()).float().double()
        h = (g / (1.0 + torch.exp(-g)) * up).float()
        d = _act(mode, h) @ _dequant(state["w_down"][i], ff).t()
        y.index_add_(0, t, gates[t, slot].double()[:, None] * d)
    return y.float()


def _run_sample(s):
    l = s["logits"].double() + 0.0
    rows, n = l.shape
    l = torch.where(torch.isnan(l), -math.inf, l)
    m = l.amax(1, keepdim=True)
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    away = torch.where(l == m, 0.0, l - m) * (1.0 / torch.where(greedy, 1.0, t))
    w = torch.floor(torch.exp(away) * UNIT + 0.5).long()
    w = torch.where(torch.isinf(l) & (l < 0), 0, w)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    w = w.gather(1, order)
    c = torch.cumsum(w, 1)
    top_k, top_p, min_p, u = (s[x][:, None] for x in ("top_k", "top_p", "min_p", "u"))
    n_k = torch.where(top_k > 0, top_k.long().clamp(max=n), n)
    w_k = c.gather(1, n_k - 1).double()
    n_p = torch.where(top_p < 1, (c.double() < top_p.double() * w_k).sum(1, keepdim=True) + 1, n)
    n_m = torch.where(min_p > 0, (w.double() >= min_p.double() * UNIT).sum(1, keepdim=True).clamp(min=1), n)
    kept = torch.minimum(torch.minimum(n_k, n_p), n_m)
    kept = torch.where(greedy, 1, kept)
    total = c.gather(1, kept - 1)
    j = torch.minimum((c.double() <= u.double() * total.double()).sum(1, keepdim=True),
                      (c < total).sum(1, keepdim=True))
    j = torch.where(greedy, 0, j)
    idx = order.gather(1, j)
    prob = w.gather(1, j).double() / total.double()
    none = torch.isinf(m) & (m < 0)
    return (torch.where(none, -1, idx).to(torch.int32).view(rows),
            torch.where(none, 0.0, prob).float().view(rows))


def run(state):
    case = state["case"]
    if own:
        q8 = state["q8"]
        if case["op"] == "sample":
            return q8.sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                             top_p=state["top_p"], min_p=state["min_p"], workspace=state["workspace"])
        if case["op"] == "moe":
            return q8.moe(state["layer"], state["x"], residual=state["residual"], workspace=state["workspace"])
        return q8.moe_experts(state["layer"], state["x"], state["ids"], state["gates"], residual=state["residual"],
                              workspace=state["workspace"])
    if case["op"] == "sample":
        return _run_sample(state)
    if case["op"] == "moe":
        ids, gates = _run_route(state, case)
        return _run_experts(state, case, ids, gates), ids, gates
    return _run_experts(state, case, state["ids"], state["gates"])


# --------------------------------------------------------------- the definition

def _exact_quant(mode, x):
    """(words as a list of f32 arrays of integers with their factor, scales) of f32 rows [m][k]."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    s = np.max(np.abs(b), axis=2) / np.float32(127)
    safe = np.where(s > 0, s, np.float32(1))[..., None]

    def rha(q):
        q = q.astype(np.float64)
        return np.clip(np.sign(q) * np.floor(np.abs(q) + 0.5), -127, 127)

    hi = np.where(s[..., None] > 0, rha(b / safe), 0.0)
    words = [(hi, 1.0)]
    if mode == "i8x2":
        rest = (b.astype(np.float64) - s[..., None].astype(np.float64) * hi).astype(np.float32)
        lo = np.where(s[..., None] > 0, rha(rest * np.float32(128) / safe), 0.0)
        words.append((lo, 1.0 / 128))
    return words, s.astype(np.float64)


def _exact_project(mode, blocks, k, x):
    """f64 [m][n] = W x for f32 rows x (numpy): block sums, then the block terms."""
    b = blocks.view(blocks.shape[0], k // BLOCK, 34)
    d = b[..., :2].contiguous().view(torch.float16).double().squeeze(-1)
    q = b[..., 2:].contiguous().view(torch.int8)
    out = []
    if mode != "f32":
        words, scales = _exact_quant(mode, x)
    for r in range(x.shape[0]):
        if mode == "f32":
            xr = torch.from_numpy(x[r].astype(np.float64)).cuda().view(-1, BLOCK)
            sums = (q.double() * xr).sum(-1)
            out.append((sums * d).sum(1))
            continue
        total = 0.0
        for word, factor in words:  # at most 32 * 127 * 127: exact in f32
            total = total + (q.float() * torch.from_numpy(word[r].astype(np.float32)).cuda()).sum(-1).double() * factor
        out.append((total * d * torch.from_numpy(scales[r]).cuda()).sum(1))
    return torch.stack(out).cpu().numpy()


def _exact_route(state, case):
    z = state["x"].double().cpu().numpy() @ state["router"].double().cpu().numpy().T
    z32 = z.astype(np.float32)
    ids = np.argsort(-z32, axis=1, kind="stable")[:, :case["top_k"]]
    p = np.exp(np.take_along_axis(z32, ids, 1).astype(np.float64))
    return ids.astype(np.int32), p / p.sum(1, keepdims=True)


def _exact_experts(state, case, ids, gates):
    x = state["x"].cpu().numpy()
    y = np.zeros(x.shape) if state["residual"] is None else state["residual"].double().cpu().numpy()
    for e in range(case["experts"]):
        pairs = np.argwhere(ids == e)
        if not len(pairs):
            continue
        rows = np.unique(pairs[:, 0])
        g = _exact_project(case["mode"], state["w_gate"][e], case["k"], x[rows]).astype(np.float32).astype(np.float64)
        up = _exact_project(case["mode"], state["w_up"][e], case["k"], x[rows]).astype(np.float32).astype(np.float64)
        h = (g / (1.0 + np.exp(-g)) * up).astype(np.float32)
        d = _exact_project(case["mode"], state["w_down"][e], case["ff"], h)
        for t, slot in pairs:
            y[t] += float(gates[t, slot]) * d[np.searchsorted(rows, t)]
    return y


def _exact_sample(s):
    idx, prob = [], []
    get = {name: s[name].cpu().numpy() for name in ("logits", "temperature", "top_k", "top_p", "min_p", "u")}
    for r in range(get["logits"].shape[0]):
        l = get["logits"][r].astype(np.float64)
        cand = np.flatnonzero(l > -np.inf)  # drops NaN too
        if not len(cand):
            idx.append(-1), prob.append(0.0)
            continue
        cand = cand[np.argsort(-l[cand], kind="stable")]
        v, temp = l[cand], float(get["temperature"][r])
        if not temp > 0:
            idx.append(cand[0]), prob.append(1.0)
            continue
        off = np.where(v == v[0], 0.0, v - v[0])
        w = np.floor(np.exp(off * (1.0 / temp)) * UNIT + 0.5).astype(np.int64)
        keep = len(w) if get["top_k"][r] <= 0 else min(len(w), int(get["top_k"][r]))
        c = np.cumsum(w)
        if get["top_p"][r] < 1:
            # f32 parameters widened, compared in f64
            keep = min(keep, int(np.count_nonzero(c < float(get["top_p"][r]) * float(c[keep - 1]))) + 1)
        if get["min_p"][r] > 0:
            keep = max(1, min(keep, int(np.count_nonzero(w >= float(get["min_p"][r]) * UNIT))))
        w, c = w[:keep], c[:keep]
        above = np.flatnonzero(c.astype(np.float64) > float(get["u"][r]) * float(c[-1]))
        j = above[0] if len(above) else np.flatnonzero(w)[-1]
        idx.append(cand[j]), prob.append(w[j] / float(c[-1]))
    return np.array(idx, np.int32), np.array(prob)


def exact(case, seed):
    state = _inputs(case, seed)
    if case["op"] == "sample":
        return _exact_sample(state)
    if case["op"] == "moe":
        ids, gates = _exact_route(state, case)
        return _exact_experts(state, case, ids, gates.astype(np.float32)), ids, gates
    return _exact_experts(state, case, state["ids"].cpu().numpy(), state["gates"].cpu().numpy())
