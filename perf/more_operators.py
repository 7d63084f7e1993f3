"""The measured cases of the key/value cache and its attention: keys and values
quantized to 4 or 8 bits as they are written into pages, read back, and attended to
by the queries of decode steps, of several rows a sequence and of prompts.

A case is a dict of plain values.  `prepare` makes its inputs on the GPU from a
seed, `run` makes one pass (the plain torch form, or the package's entry points
where `own` is true; both work on the same pages), `exact` computes the same outputs
in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TILE = 32   # tokens of one tile of a page
BLOCK = 32  # values that share a scale


# ------------------------------------------------------------------ the cases

def _case(name, op, bits, heads, kv_heads, dim, page, sequences, longest, rows=1, fresh=False, window=0, idle=0):
    """sequences: of which `idle` are empty slots of a padded batch; longest: tokens of the longest one, the
    others have fewer; rows: new rows of a sequence at most (fresh: all of its tokens are new)."""
    return {"name": name, "op": op, "bits": bits, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "sequences": sequences, "longest": longest, "rows": rows, "fresh": fresh, "window": window, "idle": idle}


def listed():
    return [
        # one new token of one sequence, written and read back: all latency
        _case("append_one_token", "append", 4, 32, 8, 128, 64, 1, 517),
        # a decode step of a padded batch, 8 bits, one key head a query head
        _case("append_batch64_8bit", "append", 8, 12, 12, 64, 32, 64, 4096, idle=4),
        # three prompts of different lengths
        _case("append_prompts", "append", 4, 32, 8, 128, 64, 3, 2048, rows=2048, fresh=True),
        # whole sequences read back (a cache that moves to another place or form)
        _case("read_sequences", "read", 4, 8, 4, 256, 64, 8, 4099, rows=4099, fresh=True),
        # one decode step of one short sequence: all latency
        _case("token_short", "attend", 4, 16, 2, 128, 64, 1, 517),
        # one decode step at the end of a very long one
        _case("token_long", "attend", 4, 32, 8, 128, 64, 1, 131071),
        # a decode step of a padded batch of sequences of all lengths
        _case("token_batch64", "attend", 4, 32, 8, 128, 64, 64, 8192, idle=4),
        # a smaller batch, 8 bits, one key head a query head
        _case("token_batch24_8bit", "attend", 8, 12, 12, 64, 32, 24, 1500),
        # drafted tokens to be verified, up to four a sequence
        _case("verify_batch16", "attend", 4, 32, 8, 128, 32, 16, 4096, rows=4),
        # a whole prompt
        _case("prompt", "attend", 4, 32, 8, 128, 64, 1, 2048, rows=2048, fresh=True),
        # chunks of two prompts after long cached parts: the largest
        _case("chunks_after_cache", "attend", 4, 32, 8, 128, 256, 2, 16384, rows=512),
        # chunks with a sliding window, 8 bits, wide heads, odd sizes
        _case("window_chunks_8bit", "attend", 8, 8, 4, 256, 64, 3, 5003, rows=700, window=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attend", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 12])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    c = {"op": op, "bits": rng.choice([4, 4, 4, 8]), "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "page": rng.choice([32, 64, 64, 128, 256]), "sequences": _log_int(rng, 1, 64), "fresh": False,
         "window": 0, "idle": 0}
    values = c["sequences"] * kv_heads * dim  # a token of every sequence
    if op != "attend":
        c["fresh"] = op == "read" or rng.random() < 0.5
        most = min(16384, (1 << 23) // values)  # a call of up to 2^23 values
        c["rows"] = _log_int(rng, 1, max(1, most)) if c["fresh"] or rng.random() < 0.5 else 1
        c["longest"] = c["rows"] if c["fresh"] else c["rows"] + _log_int(rng, 1, 4096)
    else:
        kind = rng.choice(["token", "token", "few", "rows"])
        if kind == "token":
            c["rows"], most = 1, min(131072, (1 << 28) // values)
            c["longest"] = _log_int(rng, 1, max(16, most))
        else:
            c["rows"] = rng.randint(2, 8) if kind == "few" else _log_int(rng, 16, 2048)
            c["sequences"] = min(c["sequences"], 16 if kind == "few" else 4)
            # pairs of rows and keys, and key values, as in the largest listed case or fewer
            most = min((1 << 27) * 128 // (c["sequences"] * heads * c["rows"] * dim), (1 << 27) // (c["sequences"] * kv_heads * dim))
            c["rows"] = min(c["rows"], max(16, most))
            c["fresh"] = kind == "rows" and rng.random() < 0.4
            c["longest"] = c["rows"] if c["fresh"] else c["rows"] + _log_int(rng, 1, min(32768, max(16, most)))
        if rng.random() < 0.25:
            c["window"] = _log_int(rng, 16, 2048)
    if c["rows"] == 1 and c["sequences"] > 4:
        c["idle"] = rng.choice([0, 0, 1, 4])
    return c


def _lengths(case):
    """(tokens, new rows) of each sequence: lists that the case alone decides."""
    lens, news = [], []
    for i in range(case["sequences"]):
        part = 1.0 - (0.38196601125 * i) % 1.0  # 1, then spread evenly over 0 .. 1
        n = max(1, int(round(case["longest"] * part)))
        new = n if case["fresh"] else min(n, max(1, int(round(case["rows"] * (1.0 - (0.27 * i) % 1.0)))))
        if case["sequences"] - i <= case["idle"]:
            n, new = 0, 1  # an empty slot: its row has no token
        lens.append(n)
        news.append(new)
    return lens, news


def _pairs(case):
    """Rows times the keys that they see, over all sequences."""
    total = 0
    for n, new in zip(*_lengths(case)):
        w = case["window"] or n
        for p in (range(n - new, n) if n else ()):
            total += min(p + 1, w)
    return total


def work(case):
    d, hk, h = case["dim"], case["kv_heads"], case["heads"]
    lens, news = _lengths(case)
    token = 2 * hk * d * case["bits"] // 8 + 2 * hk * (d // BLOCK) * 2  # bytes of a token in the cache
    rows = sum(news)
    if case["op"] == "append":  # f32 in, codes out and in again, f32 out
        return {"bytes": rows * (16 * hk * d + 2 * token), "flops": rows * 2 * hk * d * 8}
    if case["op"] == "read":
        return {"bytes": rows * (8 * hk * d + token), "flops": rows * 2 * hk * d * 2}
    seen = sum(min(n, (case["window"] or n) + new - 1) for n, new in zip(lens, news))
    return {"bytes": seen * token + rows * h * (8 * d + 4), "flops": 4 * d * h * _pairs(case)}


# ----------------------------------------------------------------- the inputs

def _inputs(case, seed):
    """Lengths, pages of each sequence, keys and values of every cached token, and the rows of the call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    d, hk, h, page = case["dim"], case["kv_heads"], case["heads"], case["page"]
    lens, news = _lengths(case)
    need = [(n + page - 1) // page for n in lens]
    order = torch.randperm(sum(need) + 3, device="cuda", generator=g).to(torch.int32)  # three pages of others
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    first = 0
    for i, n in enumerate(need):
        table[i, :n] = order[first:first + n].cpu()
        first += n
    # tokens one after the other: their sequence and place
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
    starts = torch.tensor([0] + lens).cumsum(0)
    pos = torch.arange(sum(lens), device="cuda") - starts.cuda()[seq]
    # keys with channels that stand out, as rotated keys have them
    k = torch.randn((len(pos), hk, d), device="cuda", generator=g)
    k *= torch.where(torch.rand((hk, d), device="cuda", generator=g) < 0.03, 6.0, 1.0)
    k += torch.randn((hk, d), device="cuda", generator=g) * 0.5
    v = torch.randn((len(pos), hk, d), device="cuda", generator=g) * 0.7
    rows = sum(news)
    # the rows of the call, as slices of one projection's output
    fused = torch.randn((rows, (h + 2 * hk) * d), device="cuda", generator=g)
    begin = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
    return {"case": dict(case), "lens": torch.tensor(lens, dtype=torch.int32).cuda(), "table": table.cuda(),
            "starts": None if case["rows"] == 1 else begin, "seq": seq, "pos": pos, "hist": (k, v), "fused": fused,
            "pages": sum(need) + 3, "capacity": (max(need) + 1) * page, "gen": g}


def _tile_bytes(case):
    return 2 * (TILE * case["dim"] * case["bits"] // 8 + TILE * case["dim"] // BLOCK * 2)


def prepare(case, seed):
    s = _inputs(case, seed)
    d, hk, h, page = case["dim"], case["kv_heads"], case["heads"], case["page"]
    # the pool, with what other sequences have left in it
    s["data"] = torch.randint(0, 256, (s["pages"], hk * (page // TILE) * _tile_bytes(case)), dtype=torch.uint8,
                              device="cuda", generator=s["gen"])
    k, v = s.pop("hist")
    where = s["table"].long()[s["seq"], s["pos"] // page]
    _store(case, s["data"], where, s["pos"] % page, *_quantize(case, k), *_quantize(case, v))
    del k, v
    fused = s["fused"]
    s["q"] = fused[:, :h * d].unflatten(1, (h, d))
    s["k"] = fused[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
    s["v"] = fused[:, (h + hk) * d:].unflatten(1, (hk, d))
    for name in ("seq", "pos", "gen"):
        del s[name]
    if own:
        import q8_projection_amd as q8
        s["q8"] = q8
        s["cache"] = q8.KVCache(case["bits"], hk, d, page, s["data"])
        s["batch"] = q8.CacheBatch(s["cache"], s["table"], s["lens"], starts=s["starts"], rows=fused.shape[0],
                                   max_rows=case["rows"])
        s["workspace"] = q8.attention_workspace(s["cache"], s["batch"], h)
    return s


# ------------------------------------------------------------- the plain form

def _quantize(case, x):
    """(codes uint8 [..][D], words int16 [..][D/32]) of f32 x [..][D]."""
    b = x.unflatten(-1, (-1, BLOCK))
    if case["bits"] == 4:
        lo, hi = b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0)
        need, drop, top = (hi.double() - lo.double()) / 15, 18, 4352.0
    else:
        need, drop, top = b.abs().amax(-1).double() / 127, 20, 512.0
    # the next number with 23 - drop mantissa bits, on binary16's subnormal grid below 2^-14
    low = 2.0 ** (drop - 37)
    up = need.float()
    up = torch.where(up.double() < need, torch.nextafter(up, torch.full_like(up, math.inf)), up)
    step = (1 << drop) - 1
    up = ((up.view(torch.int32) + step) & ~step).view(torch.float32)
    scale = torch.where(need < 2.0 ** -14, (torch.ceil(need / low) * low).float(), up).clamp(max=top)
    one = torch.where(scale == 0, torch.ones_like(scale), scale).double()[..., None]
    n = torch.round(b.double() / one)
    word = scale.half().view(torch.int16)
    if case["bits"] == 4:
        z = torch.round(-lo.double()[..., None] / one).clamp(0, 15)
        z = torch.where(scale[..., None] == 0, 0.0, z)
        n = torch.where(scale[..., None] == 0, 0.0, (n + z).clamp(0, 15))
        word = word | z[..., 0].to(torch.int16)
    else:
        n = torch.where(scale[..., None] == 0, 0.0, n.clamp(-127, 127)) + 128
    return n.to(torch.uint8).flatten(-2), word


def _places(case, page, slot):
    """Byte offsets in the pool of tokens at `slot` of `page`: (keys, key words, values, value words), each
    [tokens][kv_heads][D or D/32]."""
    d, hk, bits, dev = case["dim"], case["kv_heads"], case["bits"], page.device
    head = torch.arange(hk, device=dev)
    tile = ((page[:, None] * hk + head) * (case["page"] // TILE) + slot[:, None] // TILE) * _tile_bytes(case)
    tile, t = tile[..., None], (slot % TILE)[:, None, None]
    dim, blk = torch.arange(d, device=dev), torch.arange(d // BLOCK, device=dev)
    codes, words = TILE * d * bits // 8, TILE * (d // BLOCK) * 2
    a, b, i = t // 8, t % 4, t % 8 // 4
    keys = tile + (t * d + dim) * bits // 8
    key_words = tile + codes + (((a * 4 + b) * (d // BLOCK) + blk) * 2 + i) * 2
    if bits == 4:
        values = (((dim // 64 * 4 + a) * 16 + dim % 16) * 4 + dim // 16 % 4) * 4 + t % 8 // 2
    else:
        values = (((dim // 32 * 4 + a) * 16 + dim % 16) * 2 + dim // 16 % 2) * 8 + b * 2 + i
    value_words = tile + 2 * codes + words + ((blk * 4 + a) * 8 + b * 2 + i) * 2
    return keys, key_words, tile + codes + words + values, value_words


def _put_words(flat, at, words):
    flat[at] = (words & 255).to(torch.uint8)
    flat[at + 1] = (words >> 8 & 255).to(torch.uint8)


def _put_values(flat, at, codes, odd):
    """Codes of 4 bits into the low or (odd) the high halves of their bytes, the other halves kept."""
    flat[at] = flat[at] & 15 | codes << 4 if odd else flat[at] & 240 | codes


def _store(case, data, page, slot, k_codes, k_words, v_codes, v_words):
    flat = data.view(-1)
    keys, key_words, values, value_words = _places(case, page, slot)
    _put_words(flat, key_words, k_words)
    _put_words(flat, value_words, v_words)
    if case["bits"] == 8:
        flat[keys], flat[values] = k_codes, v_codes
        return
    flat[keys[..., ::2]] = k_codes[..., ::2] | k_codes[..., 1::2] << 4
    # two tokens share a byte of the values: the even ones are written first
    even, odd = slot % 2 == 0, slot % 2 == 1
    _put_values(flat, values[even], v_codes[even], False)
    _put_values(flat, values[odd], v_codes[odd], True)


def _values(case, codes, words):
    """f32 values of codes [..][D] and words [..][D/32]."""
    w = words[..., None]
    b = codes.unflatten(-1, (-1, BLOCK)).float()
    if case["bits"] == 4:
        return ((w & 0x7fe0).view(torch.float16).float() * (b - (w & 15).float())).flatten(-2)
    return (w.view(torch.float16).float() * (b - 128)).flatten(-2)


def _load(case, data, page, slot):
    """f32 (keys, values) [tokens][kv_heads][D]."""
    flat = data.view(-1)
    keys, key_words, values, value_words = _places(case, page, slot)
    k, v = flat[keys], flat[values]
    if case["bits"] == 4:
        high = torch.arange(case["dim"], device=flat.device) % 2 == 1
        k = torch.where(high, k >> 4, k & 15)
        v = torch.where((slot % 2 == 1)[:, None, None], v >> 4, v & 15)
    kw, vw = (flat[at].short() | flat[at + 1].short() << 8 for at in (key_words, value_words))
    return _values(case, k, kw), _values(case, v, vw)


def _rows(s):
    """(sequence, position, whether there is a token) of the call's rows."""
    case, rows = s["case"], s["fused"].shape[0]
    r = torch.arange(rows, device="cuda")
    if s["starts"] is None:
        seq, new, i = r, torch.ones_like(r), torch.zeros_like(r)
    else:
        starts = s["starts"].long()
        seq = torch.searchsorted(starts, r, right=True) - 1
        new, i = starts[seq + 1] - starts[seq], r - starts[seq]
    pos = s["lens"].long()[seq] - new + i
    return seq, i, pos, pos >= 0


def _run_append(s, write):
    case = s["case"]
    seq, _, pos, there = _rows(s)
    page = s["table"].long()[seq, pos.clamp(min=0) // case["page"]]
    slot = pos.clamp(min=0) % case["page"]
    if write:
        _store(case, s["data"], page[there], slot[there], *_quantize(case, s["k"][there]), *_quantize(case, s["v"][there]))
    k, v = _load(case, s["data"], page.clamp(min=0), slot)
    return torch.where(there[:, None, None], k, 0.0), torch.where(there[:, None, None], v, 0.0)


def _gathered(s):
    """f32 (keys, values) [sequences][kv_heads][capacity][D] of whole pages."""
    case = s["case"]
    d, hk, bits = case["dim"], case["kv_heads"], case["bits"]
    blocks = d // BLOCK
    x = s["data"][s["table"].long().clamp(min=0)]            # [S][pages][bytes]
    x = x.view(*x.shape[:2], hk, case["page"] // TILE, _tile_bytes(case)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    codes, words = TILE * d * bits // 8, TILE * blocks * 2   # [S][hk][tiles][bytes]
    kc, kw, vc, vw = x.split([codes, words, codes, words], -1)
    if bits == 4:
        k = torch.stack((kc & 15, kc >> 4), -1).flatten(-2).unflatten(-1, (TILE, d))
        v = torch.stack((vc & 15, vc >> 4), -1).flatten(-2).unflatten(-1, (d // 64, 4, 16, 4, 8))
        v = v.permute(0, 1, 2, 4, 7, 3, 6, 5)                # [g][8][D/64][i][c]
    else:
        k = kc.unflatten(-1, (TILE, d))
        v = vc.unflatten(-1, (blocks, 4, 16, 2, 4, 2)).permute(0, 1, 2, 4, 8, 7, 3, 6, 5)
    v = v.flatten(3).unflatten(-1, (TILE, d))
    kw, vw = (w.unflatten(-1, (-1, 2)) for w in (kw, vw))
    kw, vw = (w[..., 0].short() | w[..., 1].short() << 8 for w in (kw, vw))
    kw = kw.unflatten(-1, (4, 4, blocks, 2)).permute(0, 1, 2, 3, 6, 4, 5).flatten(3).unflatten(-1, (TILE, blocks))
    vw = vw.unflatten(-1, (blocks, 4, 4, 2)).permute(0, 1, 2, 4, 6, 5, 3).flatten(3).unflatten(-1, (TILE, blocks))
    return _values(case, k, kw).flatten(2, 3), _values(case, v, vw).flatten(2, 3)


def _run_attend(s):
    case = s["case"]
    d, hk, h = case["dim"], case["kv_heads"], case["heads"]
    seq, i, pos, _ = _rows(s)
    most, n, groups = case["rows"], case["sequences"], h // hk
    # rows of a sequence side by side, short ones padded with rows that see nothing
    q = torch.zeros((n, most, h, d), device="cuda")
    q[seq, i] = s["q"]
    at = torch.full((n, most), -1, device="cuda")
    at[seq, i] = pos
    q = q.view(n, most, hk, groups, d).permute(0, 2, 1, 3, 4).reshape(n, hk, most * groups, d)
    k, v = _gathered(s)
    token = torch.arange(k.shape[2], device="cuda")
    see = token <= at[..., None]
    if case["window"]:
        see &= token > at[..., None] - case["window"]
    # what lies behind a sequence's tokens may be anything
    used = (token < s["lens"][:, None])[:, None, :, None]
    k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
    score = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hk, most, groups, -1)
    score = score.masked_fill_(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(n, hk, most * groups, -1) @ v).view(n, hk, most, groups, d) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    out = out.permute(0, 2, 1, 3, 4).reshape(n, most, h, d)[seq, i]
    return out, lse.permute(0, 2, 1, 3, 4).reshape(n, most, h)[seq, i]


def run(state):
    case = state["case"]
    if own:
        q8, cache, batch = state["q8"], state["cache"], state["batch"]
        if case["op"] == "attend":
            return q8.attention(cache, batch, state["q"], window=case["window"], workspace=state["workspace"])
        if case["op"] == "append":
            q8.cache_append(cache, batch, state["k"], state["v"])
        return q8.cache_read(cache, batch)
    if case["op"] == "attend":
        return _run_attend(state)
    return _run_append(state, case["op"] == "append")


# --------------------------------------------------------------- the definition

def _exact_values(bits, x):
    """f64 values that the cache holds for x [..][D]: the scale is the smallest of the format's scales that spans
    the block (the scales are tried, not computed)."""
    b = x.double().unflatten(-1, (-1, 32))
    keep = 5 if bits == 4 else 3  # mantissa bits
    scales = torch.arange(0, 31 << 10, 1 << (10 - keep), dtype=torch.int32, device=x.device).to(torch.int16)
    scales = scales.view(torch.float16).double()
    scales = scales[scales <= (4352 if bits == 4 else 512)]
    if bits == 4:
        low, span, steps = -b.amin(-1).clamp(max=0), b.amax(-1).clamp(min=0) - b.amin(-1).clamp(max=0), 15
    else:
        low, span, steps = b.abs().amax(-1), b.abs().amax(-1), 127
    at = torch.searchsorted(scales * steps, span).clamp(max=len(scales) - 1)  # the first with scale * steps >= span
    s = scales[at][..., None]
    # quotients of numbers of 24 and 6 bits: none lies within 2^-53 of a half without being one
    n = torch.round(b / torch.where(s == 0, 1.0, s))
    if bits == 4:
        zero = torch.round(low[..., None] / torch.where(s == 0, 1.0, s)).clamp(0, 15)
        n = torch.minimum(torch.maximum(n, -zero), 15 - zero)
    else:
        n = n.clamp(-127, 127)
    return (n * s).flatten(-2)


def exact(case, seed):
    s = _inputs(case, seed)
    hk, h, d, bits = case["kv_heads"], case["heads"], case["dim"], case["bits"]
    lens, news = _lengths(case)
    # what prepare() draws between the inputs does not touch the rows of the call
    fused = s["fused"]
    if case["op"] == "append":
        there = torch.cat([torch.arange(n - new, n) >= 0 for n, new in zip(lens, news)]).cuda()[:, None, None]
        return tuple(torch.where(there, _exact_values(bits, x.unflatten(1, (hk, d))), 0.0)
                     for x in (fused[:, h * d:(h + hk) * d], fused[:, (h + hk) * d:]))
    hk_all, hv_all = s.pop("hist")
    if case["op"] == "read":  # every token is a row
        return _exact_values(bits, hk_all), _exact_values(bits, hv_all)
    outs, lses, first, row = [], [], 0, 0
    for n, new in zip(lens, news):
        q = fused[row:row + new, :h * d].double().view(new, hk, h // hk, d)
        row += new
        k, v = (_exact_values(bits, x[first:first + n]).transpose(0, 1) for x in (hk_all, hv_all))  # [hk][n][d]
        first += n
        out, lse = torch.zeros((new, h, d), dtype=torch.float64), torch.full((new, h), -math.inf, dtype=torch.float64)
        for r0 in range(0, new if n else 0, 128):
            r1 = min(new, r0 + 128)
            p = torch.arange(n - new + r0, n - new + r1, device="cuda")[:, None]
            t0 = max(0, n - new + r0 + 1 - case["window"]) if case["window"] else 0
            t1 = n - new + r1
            t = torch.arange(t0, t1, device="cuda")
            see = (t <= p) & (t > p - (case["window"] or n))
            z = torch.matmul(q[r0:r1].permute(1, 2, 0, 3).reshape(hk, -1, d), k[:, t0:t1].transpose(1, 2).contiguous())
            z = (z / math.sqrt(d)).view(hk, h // hk, r1 - r0, -1).masked_fill(~see, -math.inf)
            e = torch.logsumexp(z, -1)
            o = torch.matmul(torch.exp(z - e[..., None]).flatten(1, 2), v[:, t0:t1].contiguous())
            out[r0:r1] = o.view(hk, h // hk, r1 - r0, d).permute(2, 0, 1, 3).reshape(r1 - r0, h, d).cpu()
            lse[r0:r1] = e.permute(2, 0, 1).reshape(r1 - r0, h).cpu()
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs).cuda(), torch.cat(lses).cuda()
