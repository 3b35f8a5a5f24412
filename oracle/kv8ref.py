"""Float64 oracle of the 8-bit paged KV cache (include/apr_kv8.h).

Plain loops over sequences, heads and pages; nothing is shared with the CUDA
library. A cache is a dict of numpy arrays: K, V int8 [pages][heads][tokens][dim],
k_scale, v_scale float32 [pages][heads]; table, lens and row_start are integer
arrays (row_start None: one row a sequence). Functions that write the cache
return a changed copy.
"""

from __future__ import annotations

import math

import numpy as np


def kv8_scale(amax):
    """float32(amax / 127) of a float32 magnitude."""
    return np.float32(np.float64(amax) / 127.0)


def kv8_codes(x, scale):
    """Codes of float32 values: nearest whole number to x / scale (ties to even), clamped to +-127; NaN 0, infinities
    +-127; 0 under scale 0. The float64 quotient of two float32 numbers is on the exact quotient's side of every half."""
    x = np.asarray(x, np.float32)
    s = np.float64(scale)
    if not s > 0:
        return np.zeros(x.shape, np.int8)
    with np.errstate(invalid="ignore"):
        r = np.clip(np.rint(x.astype(np.float64) / s), -127, 127)
    return np.where(np.isnan(x), 0, r).astype(np.int8)


def kv8_values(codes, scale):
    """float32 values code * scale."""
    return codes.astype(np.float32) * np.float32(scale)


def _spans(lens, row_start):
    """(sequence, first packed row, rows, length) of each sequence."""
    for b, n in enumerate(lens):
        r0, r1 = (b, b + 1) if row_start is None else (int(row_start[b]), int(row_start[b + 1]))
        yield b, r0, r1 - r0, int(n)


def kv8_append(cache, table, lens, row_start, k, v):
    new = {name: a.copy() for name, a in cache.items()}
    heads, tokens = cache["K"].shape[1:3]
    for b, r0, n, length in _spans(lens, row_start):
        first = length - n
        for index in range(max(first, 0) // tokens, -(-length // tokens)):
            lo, hi = max(first, 0, index * tokens), min(length, (index + 1) * tokens)
            if lo >= hi:
                continue
            page, held = table[b][index], lo - index * tokens
            for name, rows in (("K", k), ("V", v)):
                codes, scales = new[name], new[name.lower() + "_scale"]
                for g in range(heads):
                    x = np.asarray(rows, np.float32).reshape(len(rows), heads, -1)[r0 + lo - first:r0 + hi - first, g]
                    finite = np.abs(x[np.isfinite(x)])
                    old = scales[page, g] if held else np.float32(0)
                    s = max(old, kv8_scale(finite.max() if finite.size else 0.0))
                    if s > old:
                        codes[page, g, :held] = kv8_codes(kv8_values(codes[page, g, :held], old), s)
                    codes[page, g, held:held + hi - lo] = kv8_codes(x, s)
                    scales[page, g] = s
    return new


def kv8_read(cache, table, lens, row_start, rows):
    """(k, v) float32 [rows][heads][dim]; rows before a sequence's start are 0."""
    heads, tokens, dim = cache["K"].shape[1:]
    k, v = (np.zeros((rows, heads, dim), np.float32) for _ in range(2))
    for b, r0, n, length in _spans(lens, row_start):
        for i in range(n):
            pos = length - n + i
            if pos >= 0:
                page, slot = table[b][pos // tokens], pos % tokens
                k[r0 + i] = kv8_values(cache["K"][page, :, slot], cache["k_scale"][page][:, None])
                v[r0 + i] = kv8_values(cache["V"][page, :, slot], cache["v_scale"][page][:, None])
    return k, v


def _whole(cache, name, table_row, length):
    """float64 values [heads][length][dim] of a sequence."""
    heads, tokens, dim = cache[name].shape[1:]
    pages = list(table_row[: -(-length // tokens)])
    x = cache[name][pages].astype(np.float64) * cache[name.lower() + "_scale"][pages].astype(np.float64)[..., None, None]
    return x.transpose(1, 0, 2, 3).reshape(heads, len(pages) * tokens, dim)[:, :length]


def kv8_attention(cache, table, lens, row_start, q, num_heads, scale=0.0):
    """(out [rows][num_heads][dim], weights [sequences][kv_heads][max length], reach [rows][num_heads]) in float64;
    reach is the largest sum of |scale q_c k_c| over a position that the row sees."""
    kv, _, dim = cache["K"].shape[1:]
    group = num_heads // kv
    q = np.asarray(q, np.float64).reshape(-1, num_heads, dim)
    out, reach = np.zeros(q.shape), np.zeros(q.shape[:2])
    weights = np.zeros((len(lens), kv, max([int(n) for n in lens] + [0])))
    factor = scale if scale else 1.0 / math.sqrt(dim)
    for b, r0, n, length in _spans(lens, row_start):
        if not length or not n:
            continue
        K, V = _whole(cache, "K", table[b], length), _whole(cache, "V", table[b], length)
        for i in range(n):
            sees = length - n + i + 1
            if sees <= 0:
                continue
            for h in range(num_heads):
                g = h // group
                s = K[g, :sees] @ q[r0 + i, h] * factor
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r0 + i, h] = p @ V[g, :sees]
                weights[b, g, :sees] += p
                reach[r0 + i, h] = (np.abs(K[g, :sees]) @ np.abs(q[r0 + i, h])).max() * factor
    return out, weights, reach


def kv8_evict(cache, table, lens, weights, budget, recent, fresh):
    """(cache, table_out, lens_out, weights_out, kept)."""
    new = {name: a.copy() for name, a in cache.items()}
    heads, tokens, dim = cache["K"].shape[1:]
    count = len(lens)
    table_out = np.full(np.shape(table), -1, np.int32)
    lens_out = np.minimum(np.asarray(lens), budget).astype(np.int32)
    weights_out = np.zeros((count, heads, budget), np.float32)
    kept = np.full((count, heads, budget), -1, np.int32)
    for b in range(count):
        length, now = int(lens[b]), int(lens_out[b])
        pages = -(-now // tokens)
        table_out[b, :pages] = (fresh if length > budget else table)[b][:pages]
        for g in range(heads):
            w = np.asarray(weights[b][g][:length], np.float32)
            if length > budget:
                old = length - recent
                rank = np.where(np.isnan(w[:old]), np.inf, w[:old].astype(np.float64))
                best = sorted(range(old), key=lambda j: (not np.isnan(w[j]), -rank[j], j))[:budget - recent]
                pick = np.array(sorted(best) + list(range(old, length)), np.int64)
            else:
                pick = np.arange(length)
            kept[b, g, :now], weights_out[b, g, :now] = pick, w[pick]
            if length <= budget:
                continue
            for name in ("K", "V"):
                scales = cache[name.lower() + "_scale"]
                rows = np.stack([kv8_values(cache[name][table[b][j // tokens], g, j % tokens],
                                            scales[table[b][j // tokens], g]) for j in pick])
                for i in range(pages):
                    x = rows[i * tokens:(i + 1) * tokens]
                    s = kv8_scale(np.abs(x).max())
                    new[name.lower() + "_scale"][fresh[b][i], g] = s
                    new[name][fresh[b][i], g, : len(x)] = kv8_codes(x, s)
    return new, table_out, lens_out, weights_out, kept
