"""Oracle of the block-sparse decode attention: bounds of blocks, the selection by them, and
the attention over what is selected; numpy in 64 bits and whole numbers."""
from __future__ import annotations

import math

import numpy as np


def exponent(most):
    """The least e >= -50 with most <= 127 * 2^e; 51 where there is none up to 50."""
    if not most <= 127 * 2.0 ** 50:  # a NaN too
        return 51
    e = -50
    while most > 127 * 2.0 ** e:
        e += 1
    return e


def tile_bounds(keys):
    """int8 [2, D] and the scale of keys [tokens, D] of one (block, KV head)."""
    keys = np.asarray(keys, dtype=np.float64)
    out = np.zeros((2, keys.shape[1]), dtype=np.int8)
    e = exponent(math.nan if np.isnan(keys).any() else np.abs(keys).max())
    if e > 50:
        return out, math.inf
    out[0] = np.ceil(keys.max(0) / 2.0 ** e)
    out[1] = np.floor(keys.min(0) / 2.0 ** e)
    return out, 2.0 ** e


def block_bounds(bounds, scales, k_cache, block_tables, context_lens, new_tokens, max_new):
    """Writes the bounds (numpy int8 [NB, Hkv, 2, D]) and scales of the blocks that hold new
    tokens; returns the status bits."""
    nb, hkv, block, _ = k_cache.shape
    status = 0
    for s, (length, new) in enumerate(zip(context_lens, new_tokens)):
        if new <= 0:
            continue
        if length < new or new > max_new or length > len(block_tables[s]) * block:
            status |= 2
            continue
        for j in range((length - new) // block, -(-length // block)):
            b = block_tables[s][j]
            if not 0 <= b < nb:
                status |= 1
                continue
            for h in range(hkv):
                bounds[b, h], scales[b, h] = tile_bounds(k_cache[b, h, :length - j * block])
    return status


def quantise_query(row):
    """Whole numbers in -127 .. 127 and their unit of a query row."""
    row = np.asarray(row, dtype=np.float64)
    row = np.where(np.isnan(row), 0.0, row)
    unit = 2.0 ** min(50, exponent(np.abs(row).max()))
    with np.errstate(invalid="ignore"):
        return np.clip(np.floor(row / unit + 0.5), -127, 127), unit


def block_scores(q, bounds, scales):
    """Scores of blocks (bounds [n, 2, D], scales [n]) for the query rows q [G, D]."""
    best = np.full(len(scales), -math.inf)
    wide = bounds.astype(np.float64)
    for row in q:
        c, unit = quantise_query(row)
        best = np.maximum(best, (np.maximum(c, 0) * wide[:, 0] + np.minimum(c, 0) * wide[:, 1])
                          .sum(-1) * unit)
    with np.errstate(invalid="ignore"):
        return np.where(np.isinf(scales), math.inf, best * scales)


def select(q, bounds, scales, block_tables, context_lens, block, k, first=1, recent=1,
           scores=None):
    """(selected [S, Hkv, K], selected_lens [S, Hkv], scores [S, Hkv, width], status) of query
    rows q [S, Hq, D]; scores keeps its values where nothing is written."""
    S, heads, _ = np.asarray(q).shape
    nb, hkv = scales.shape
    width = len(block_tables[0])
    group = heads // hkv
    selected = np.full((S, hkv, k), -1, dtype=np.int32)
    lens = np.zeros((S, hkv), dtype=np.int32)
    scores = np.zeros((S, hkv, width)) if scores is None else scores.copy()
    status = 0
    for s in range(S):
        length = int(context_lens[s])
        if length < 0 or length > width * block:
            status |= 2
            length = 0
        n = -(-length // block)
        ids = np.array([int(b) for b in block_tables[s][:n]], dtype=np.int64)
        good = (ids >= 0) & (ids < nb)
        at = np.where(good, ids, 0)
        for h in range(hkv):
            if n <= k:
                keep = list(range(n))
                scores[s, h, :n] = math.inf
            else:
                row = block_scores(q[s][h * group:(h + 1) * group], bounds[at, h], scales[at, h])
                row = np.where(good, row, -math.inf)
                middle = sorted(range(first, n - recent), key=lambda i: (-row[i], i))
                keep = sorted(list(range(first)) + list(range(n - recent, n)) +
                              middle[:k - first - recent])
                row[:first] = row[n - recent:] = math.inf
                scores[s, h, :n] = row
                if not good[first:n - recent].all():
                    status |= 1
            for i, b in enumerate(keep):
                selected[s, h, i] = ids[b] * hkv + h if good[b] else -1
                status |= 0 if good[b] else 1
            lens[s, h] = sum(min(block, length - b * block) for b in keep)
    return selected, lens, scores, status


def attention(q, k_cache, v_cache, selected, selected_lens, scale):
    """out [S, Hq, D] in float64 over caches [NB, Hkv, B, D]; a tile outside them hides its
    tokens, no token gives a row of zeros."""
    q = np.asarray(q, dtype=np.float64)
    S, heads, d = q.shape
    nb, hkv, block, _ = k_cache.shape
    group = heads // hkv
    keys, values = (np.asarray(c).reshape(nb * hkv, block, d) for c in (k_cache, v_cache))
    out = np.zeros((S, heads, d))
    for s in range(S):
        for h in range(hkv):
            n = int(selected_lens[s][h])
            ids = np.asarray(selected[s][h][:-(-n // block)], dtype=np.int64)
            good = (ids >= 0) & (ids < nb * hkv)
            seen = np.repeat(good, block)[:n]
            if not seen.any():
                continue
            ids = np.where(good, ids, 0)
            k, v = (c[ids].reshape(-1, d)[:n][seen].astype(np.float64) for c in (keys, values))
            rows = slice(h * group, (h + 1) * group)
            x = q[s, rows] @ k.T * scale
            p = np.exp(x - x.max(-1, keepdims=True))
            out[s, rows] = p @ v / p.sum(-1, keepdims=True)
    return out
