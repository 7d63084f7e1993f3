"""The key/value cache and its attention in 64 bits, from the formulas of
include/q8_cache.h (numpy; nothing of the library).

Bound of the attention's outputs.  With Z the largest sum_j |q_j k_tj| * |scale| over the
tokens that a row sees, and A = sum_t p_t |v_t| of its outputs:
  a score is off by at most  ez = Z (2^-21 + (D + 8) 2^-24) + 8 * 2^-24 (1 + |z| max)
      q in two binary16 words: each at most half a step of 11 bits off, 2^-12 * 2^-12 together
      with the rounding of scale and q: under 2^-21; D products added in f32: at most D + 8
      roundings; the scale's, the difference's and the exponential's roundings
  a weight p_t is then off by 2 ez + 2^-21 (two words), relative, ez for the sum's as well
  a weight is also off by 2^-36 of the largest one, absolute: its words lie on binary16's grid of
      2^-24 (half a step: 2^-25) where the largest is 2^11 or more (and f32 exponentials vanish under 2^-149)
  sums over the tokens are added in f32 in chains: at most (T / 8 + 64) 2^-24, relative to A
so |out - ref| <= A (2 ez + 2^-20 + (T / 8 + 64) 2^-24) + 2^-36 sum_t |v_t| / sum_t exp(z_t - max z), and lse
is off by
ez + (T / 8 + 64) 2^-24 + 2^-23 |lse| at most.

Roundings that do not all point the same way add up as their squares do.  D + 8 of them, none
over 2^-24 Z, then make sqrt(D + 8) 2^-24 Z of a score, with 4 * 2^-24 |z| max for the scale's,
the difference's and the exponential's; and T of them sqrt(T) 2^-24 of a sum.  The 2-norm of the
outputs' errors is held to that of A (2 ez' + 2^-20 + sqrt(T) 2^-24), ez' = 2^-24 (sqrt(D + 8) Z +
4 (1 + |z| max)).  (A score of 1000 cannot be nearer than 2^-15 in f32: no fixed part of the
output's norm would do.)
"""
from __future__ import annotations

import numpy as np

TOP = {4: 4352.0, 8: 512.0}


def scales(bits):
    """Every scale of the format, ascending from 0."""
    low = 5 if bits == 4 else 7
    s = np.arange(0, 0x7c00, 1 << low, dtype=np.uint16).view(np.float16).astype(np.float64)
    return s[s <= TOP[bits]]


def quantize(bits, x):
    """(codes int [..][D], scales f64 [..][D/32], zero points int [..][D/32]) of f32 x [..][D]."""
    b = x.astype(np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    lo, hi = np.minimum(b.min(-1), 0), np.maximum(b.max(-1), 0)
    all_scales = scales(bits)
    steps = 15 if bits == 4 else 127
    span = hi - lo if bits == 4 else np.maximum(hi, -lo)
    d = all_scales[np.minimum(np.searchsorted(all_scales * steps, span), len(all_scales) - 1)]
    one = np.where(d == 0, 1.0, d)
    # (f64 quotients of 24-bit by 6-bit numbers are a half-integer only where the exact ones are)
    n = np.where(d[..., None] == 0, 0.0, np.rint(b / one[..., None]))
    if bits == 4:
        z = np.where(d == 0, 0.0, np.minimum(np.rint(-lo / one), 15.0))
        n = np.clip(n + z[..., None], 0, 15)
    else:
        z = np.zeros_like(d)
        n = np.clip(n, -127, 127)
    return n.reshape(x.shape).astype(np.int64), d, z.astype(np.int64)


def values(bits, x):
    """f64 values that the cache stands for (binary16 numbers)."""
    n, d, z = quantize(bits, x)
    n = n.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    return ((n - z[..., None]) * d[..., None]).reshape(x.shape)


def tile_parts(bits, d):
    """Byte offsets of the parts of a tile and its size."""
    codes, words = 32 * d * bits // 8, 32 * (d // 32) * 2
    return 0, codes, codes + words, 2 * codes + words, 2 * (codes + words)


def pack(bits, k, v, tile):
    """Write 32 tokens' keys and values [32][D] into the bytes of a tile (uint8), by the layout's formulas."""
    d = k.shape[1]
    kc, kw, vc, vw, size = tile_parts(bits, d)
    assert tile.shape == (size,)
    words = np.zeros((2, 32, d // 32), np.uint16)
    codes = np.zeros((2, 32, d), np.int64)
    for which, x in enumerate((k, v)):
        n, s, z = quantize(bits, x)
        codes[which] = n if bits == 4 else n + 128
        words[which] = s.astype(np.float16).view(np.uint16) | (z.astype(np.uint16) if bits == 4 else 0)

    def put(base, index, code):  # code number `index` of an array of codes
        if bits == 8:
            tile[base + index] = code
        else:
            at, shift = base + index // 2, 4 * (index % 2)
            tile[at] = int(tile[at]) & (255 - (15 << shift)) | code << shift

    for t in range(32):
        a, b, i = t // 8, t % 4, t % 8 // 4
        for dim in range(d):
            put(kc, t * d + dim, int(codes[0, t, dim]))
            w, c = dim // 16, dim % 16
            if bits == 4:
                put(vc, (((w // 4 * 4 + a) * 16 + c) * 4 + w % 4) * 8 + t % 8, int(codes[1, t, dim]))
            else:
                put(vc, ((((w // 2 * 4 + a) * 16 + c) * 2 + w % 2) * 4 + b) * 2 + i, int(codes[1, t, dim]))
        for blk in range(d // 32):
            for base, index, word in ((kw, ((a * 4 + b) * (d // 32) + blk) * 2 + i, words[0, t, blk]),
                                      (vw, ((blk * 4 + a) * 4 + b) * 2 + i, words[1, t, blk])):
                tile[base + 2 * index] = int(word) & 255
                tile[base + 2 * index + 1] = int(word) >> 8


def attend(q, k, v, at, scale, window=0, have=None):
    """(out, lse, bound of out, bound of lse, usual error of out) of f64 queries [rows][heads][D] at tokens `at` over values k, v
    [tokens][kv_heads][D]; have: tokens that there are (None: all)."""
    rows, heads, d = q.shape
    kv_heads = k.shape[1]
    t = np.arange(k.shape[0])
    out, lse = np.zeros(q.shape), np.full((rows, heads), -np.inf)
    out_bound, lse_bound, usual = np.zeros(q.shape), np.zeros((rows, heads)), np.zeros(q.shape)
    for r in range(rows):
        see = t <= at[r]
        if window:
            see &= t > at[r] - window
        if have is not None:
            see &= have
        if not see.any():
            continue
        ks, vs = k[see], v[see]
        for h in range(heads):
            kh, vh = ks[:, h // (heads // kv_heads)], vs[:, h // (heads // kv_heads)]
            z = scale * (kh @ q[r, h])
            most = np.abs(scale) * (np.abs(kh) @ np.abs(q[r, h])).max()
            top = z.max()
            e = np.exp(z - top)
            out[r, h] = (e / e.sum()) @ vh
            lse[r, h] = top + np.log(e.sum())
            ez = most * (2.0 ** -21 + (d + 8) * 2.0 ** -24) + 8 * 2.0 ** -24 * (1 + np.abs(z).max())
            chain = (len(z) / 8 + 64) * 2.0 ** -24
            size = (e / e.sum()) @ np.abs(vh)
            out_bound[r, h] = size * (2 * ez + 2.0 ** -20 + chain) + 2.0 ** -36 * np.abs(vh).sum(0) / e.sum()
            usual[r, h] = size * (2.0 ** -23 * (np.sqrt(d + 8) * most + 4 * (1 + np.abs(z).max())) + 2.0 ** -20 +
                                  np.sqrt(len(z)) * 2.0 ** -24)
            lse_bound[r, h] = ez + chain + 2.0 ** -23 * abs(lse[r, h])
    return out, lse, out_bound, lse_bound, usual
