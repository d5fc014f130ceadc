"""Oracle of the 4-bit KV cache: numpy in 64 bits, taken apart byte by byte.

A pool is uint8 [NB, Hkv, B, 9 * D / 16]; its last two dimensions are one tile:
B * D / 2 bytes of codes, then for every token and run of 64 elements the pair
(scale, minimum) in the cache's 16-bit type.  An element stands for
minimum + code * scale.
"""
from __future__ import annotations

import numpy as np
import torch

RUN = 64


def quantise(x: torch.Tensor):
    """Codes uint8 [..., D] and (scale, minimum) in x's 16-bit type
    [..., D / 64, 2] of rows x [..., D]."""
    lead, d = x.shape[:-1], x.shape[-1]
    runs = x.reshape(*lead, d // RUN, RUN)
    wide = runs.to(torch.float64).numpy()
    with np.errstate(all="ignore"):
        least, most = wide.min(-1), wide.max(-1)
        spread = (most - least).astype(np.float32)  # 16-bit values: the difference, rounded once
        # the quotient in 32 bits, then the 16-bit type
        scale16 = torch.from_numpy(spread / np.float32(15)).to(x.dtype)
        scale = scale16.to(torch.float64).numpy()
        ratio = (wide - least[..., None]) / np.where(scale > 0, scale, np.inf)[..., None]
        codes = np.clip(np.floor(ratio + 0.5), 0, 15)
    bad = ~np.isfinite(spread)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    low = torch.from_numpy(np.where(bad, np.nan, least)).to(x.dtype)
    scale16 = torch.where(torch.from_numpy(bad), torch.full_like(scale16, float("nan")), scale16)
    return codes.reshape(*lead, d), torch.stack([scale16, low], dim=-1)


def code_place(i: int, e, block: int, d: int, is_v: bool):
    """Byte and shift of element e of token i in a tile."""
    if is_v:
        return i // 2 * d + e // 4 * 4 + i % 2 * 2 + e % 4 // 2, 4 * (e % 2)
    return i * (d // 2) + e // 2, 4 * (e % 2)


def pair_place(i: int, block: int, d: int) -> slice:
    """Bytes of token i's pairs in a tile."""
    start = block * d // 2 + i * (d // RUN) * 4
    return slice(start, start + (d // RUN) * 4)


def kv_write(k_pool, v_pool, key, value, slot_mapping):
    """Quantises key / value [T, Hkv, D] into the pools (CPU, in place)."""
    nb, hkv, block, _ = k_pool.shape
    d = key.shape[2]
    for pool, rows, is_v in ((k_pool, key, False), (v_pool, value, True)):
        tiles = pool.view(nb, hkv, -1).numpy()
        codes, pairs = quantise(rows)
        words = pairs.contiguous().view(torch.uint8).reshape(rows.shape[0], hkv, -1).numpy()
        even, odd = np.arange(0, d, 2), np.arange(1, d, 2)
        for t, slot in enumerate(slot_mapping.tolist()):
            if slot < 0 or slot >= nb * block:
                continue
            b, i = slot // block, slot % block
            at, _ = code_place(i, even, block, d, is_v)
            tiles[b][:, at] = codes[t][:, even] | (codes[t][:, odd] << 4)
            tiles[b][:, pair_place(i, block, d)] = words[t]


def values(pool: torch.Tensor, d: int, dtype: torch.dtype, is_v: bool) -> np.ndarray:
    """What every slot of a pool stands for: float64 [NB, Hkv, B, D]."""
    nb, hkv, block, _ = pool.shape
    tiles = pool.reshape(nb, hkv, -1).contiguous()
    raw = tiles.numpy()
    out = np.empty((nb, hkv, block, d))
    e = np.arange(d)
    for i in range(block):
        at, shift = code_place(i, e, block, d, is_v)
        codes = (raw[:, :, at] >> shift) & 15
        pairs = tiles[:, :, pair_place(i, block, d)].contiguous().view(dtype)
        pairs = pairs.to(torch.float64).numpy().reshape(nb, hkv, d // RUN, 2)
        out[:, :, i] = np.repeat(pairs[..., 1], RUN, -1) + codes * np.repeat(pairs[..., 0], RUN, -1)
    return out


def kv_read(k_pool, v_pool, slot_mapping, d, dtype):
    """float64 rows [T, Hkv, D] of K and V; NaN rows for slots outside the pool."""
    block = k_pool.shape[2]
    slots = np.asarray(slot_mapping, dtype=np.int64)
    inside = (slots >= 0) & (slots < k_pool.shape[0] * block)
    at = np.where(inside, slots, 0)
    out = []
    for pool, is_v in ((k_pool, False), (v_pool, True)):
        rows = values(pool, d, dtype, is_v)[at // block, :, at % block]
        rows[~inside] = np.nan
        out.append(rows)
    return out


def paged_decode_attention(q, k_pool, v_pool, block_tables, context_lens, scale, dtype=None):
    """out[s, h] = sum_i softmax_i(scale q . k_i) v_i in float64; a table entry
    outside the pool hides its tokens, a context of no tokens gives zeros."""
    S, heads, d = q.shape
    nb, hkv, block, _ = k_pool.shape
    dtype = dtype or q.dtype
    K, V = values(k_pool, d, dtype, False), values(v_pool, d, dtype, True)
    group = heads // hkv
    wide = q.to(torch.float64).numpy()
    out = np.zeros((S, heads, d))
    for s in range(S):
        n = int(context_lens[s])
        ids = np.array([int(x) for x in block_tables[s][:-(-n // block)]], dtype=np.int64)
        seen = np.repeat((ids >= 0) & (ids < nb), block)[:n]
        ids = np.where((ids >= 0) & (ids < nb), ids, 0)
        if not seen.any():
            continue
        for g in range(hkv):
            k = K[ids, g].reshape(-1, d)[:n][seen]
            v = V[ids, g].reshape(-1, d)[:n][seen]
            x = wide[s, g * group:(g + 1) * group] @ k.T * scale
            p = np.exp(x - x.max(-1, keepdims=True))
            out[s, g * group:(g + 1) * group] = p @ v / p.sum(-1, keepdims=True)
    return out
