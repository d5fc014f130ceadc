"""The 4-bit KV cache and the GPU block tables: cases, plain forms, exact results.

Four kinds of case, one for each way in which a serving loop uses the operators:

attend    one query token per sequence attends over a paged cache held in 4 bits
store     new tokens' K and V are quantised into their slots and read back
load      the K and V of any set of slots are read back as 16-bit rows
extend    block tables, slot map and positions of a step from its request lengths
turnover  a batch of requests is admitted (extend) and then released

The 4-bit pools are uint8 [num_blocks][kv_heads][block][9 * head_dim / 16].  The last two
dimensions are one tile: first block * head_dim / 2 bytes of codes, then, for every token and
every 64 elements of head_dim, the pair (scale, minimum) in the cache's 16-bit type.  An element
stands for minimum + code * scale.
  K codes: the row of token i is head_dim / 2 bytes, element 2b in the low half of byte b and
  element 2b + 1 in its high half.
  V codes: tokens 2p and 2p + 1 share head_dim bytes of 4-byte words; word j holds elements
  4j .. 4j + 3 of token 2p in its first two bytes and those of token 2p + 1 in its last two.
A row is quantised in runs of 64: minimum = the least value, scale = (greatest - least) / 15
rounded to the 16-bit type, code = floor((x - minimum) / scale + 1/2) held to 0 .. 15.
"""
import math
import random

import numpy as np
import torch

#: False: the plain forms below; True: the framework's kernels.
own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
RUN = 64  # elements of a row that share a scale and a minimum
DEV = "cuda"


# ---- cases ---------------------------------------------------------------------------------

def _attend(name, dtype, heads, kv_heads, head_dim, block, seqs, lens, lo, hi, partition=0,
            plan=False):
    return dict(name=name, op="attend", dtype=dtype, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, block=block, seqs=seqs, lens=lens, lo=lo, hi=hi,
                partition=partition, plan=plan)


def listed():
    return [
        # four short chats on a small model: the call is all latency
        _attend("attend-4seq-d64", "f16", 8, 4, 64, 8, 4, "uniform", 1, 160),
        # one request alone with a long document: few rows, split over the GPU
        _attend("attend-1x16384-split", "bf16", 64, 4, 128, 16, 1, "fixed", 16384, 16384, 256),
        # the decode step of a multi-head model, ragged contexts up to 2048
        _attend("attend-mha32-64seq", "bf16", 32, 32, 128, 16, 64, "uniform", 1, 2048, 0, True),
        # a large grouped-query batch, lognormal context lengths, longest first
        _attend("attend-gqa64x8-256seq", "bf16", 64, 8, 128, 16, 256, "lognormal", 16, 4096, 0,
                True),
        # eight long contexts, each split in partitions of 512 tokens
        _attend("attend-gqa32x8-8x32768", "bf16", 32, 8, 128, 32, 8, "fixed", 32768, 32768, 512),
        # the new tokens of one decode step of 64 sequences, rows of a fused projection
        dict(name="store-step-64", op="store", dtype="bf16", kv_heads=32, head_dim=128, block=16,
             tokens=64, scattered=True, fused=True),
        # a batch of prompts, 32768 tokens in all
        dict(name="store-prompts-32768", op="store", dtype="f16", kv_heads=8, head_dim=128,
             block=16, tokens=32768, scattered=False, fused=False),
        # a cached history brought back to 16 bits for a prompt chunk that attends over it
        dict(name="load-history-40961", op="load", dtype="bf16", kv_heads=8, head_dim=128,
             block=32, tokens=40961),
        # a decode step: one new token for each of 64 sequences
        dict(name="extend-step-64", op="extend", seqs=64, block=16, lo=1, hi=2048, new_lo=1,
             new_hi=1, pad=0),
        # a mixed step: 1000 requests, each with up to 1024 prompt tokens, padded rows
        dict(name="extend-mixed-1000", op="extend", seqs=1000, block=8, lo=0, hi=4096, new_lo=0,
             new_hi=1024, pad=777),
        # a handful of short prompts admitted, and released when they are done
        dict(name="turnover-9", op="turnover", seqs=9, block=32, lo=1, hi=300),
        # a wave of 256 prompts
        dict(name="turnover-256", op="turnover", seqs=256, block=16, lo=16, hi=4096),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "store", "load", "extend", "turnover"])
    dtype, block = rng.choice(["bf16", "f16"]), rng.choice([8, 16, 32])
    head_dim = rng.choice([64, 128, 128])
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
        seqs = _spread(rng, 1, 256)
        # at most the cache rows of the largest listed case
        most = max(1, 8 * 8 * 32768 // (seqs * kv_heads * max(1, group // 8)))
        hi = _spread(rng, 1, min(32768, most))
        lens = rng.choice(["fixed", "uniform", "uniform", "lognormal"])
        split = rng.choice([0, 0, 1])
        return dict(op=op, dtype=dtype, heads=group * kv_heads, kv_heads=kv_heads,
                    head_dim=head_dim, block=block, seqs=seqs, lens=lens,
                    lo=hi if lens == "fixed" else rng.randint(0, hi), hi=hi,
                    partition=split * 32 * rng.randint(4, 32), plan=rng.random() < 0.6)
    if op == "store":
        return dict(op=op, dtype=dtype, kv_heads=rng.randint(1, 8), head_dim=head_dim, block=block,
                    tokens=_spread(rng, 1, 32768), scattered=rng.random() < 0.5,
                    fused=rng.random() < 0.5)
    if op == "load":
        return dict(op=op, dtype=dtype, kv_heads=rng.randint(1, 8), head_dim=head_dim, block=block,
                    tokens=_spread(rng, 1, 40961))
    if op == "extend":
        hi, new = _spread(rng, 1, 4096), _spread(rng, 1, 1024)
        return dict(op=op, seqs=_spread(rng, 1, 1000), block=block, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, new), new_hi=new, pad=rng.randint(0, 999))
    hi = _spread(rng, 1, 4096)
    return dict(op=op, seqs=_spread(rng, 1, 256), block=block, lo=rng.randint(0, hi), hi=hi)


def _lengths(case):
    """The requests' lengths: of the case alone, so that its work is known."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    rng = np.random.default_rng([n, lo, hi, case["block"]])
    if case.get("lens") == "fixed":
        return np.full(n, hi, dtype=np.int64)
    if case.get("lens") == "lognormal":
        return np.clip(np.exp(rng.normal(math.log(max(hi, 2)) - 2.0, 0.8, n)), lo, hi).astype(np.int64)
    return rng.integers(lo, hi + 1, n)


def _new_tokens(case):
    if case["op"] == "turnover":
        return _lengths(case)
    rng = np.random.default_rng([case["seqs"], case["new_lo"], case["new_hi"]])
    return rng.integers(case["new_lo"], case["new_hi"] + 1, case["seqs"])


def _blocks(n, block):
    return -(-n // block)


# ---- inputs --------------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _tables(lens, block, rng):
    """Block tables over a shuffled pool a quarter larger than need be, -1 behind the last block."""
    need = _blocks(lens, block)
    total = int(need.sum())
    order = rng.permutation(max(1, math.ceil(1.25 * total))).astype(np.int32)
    start = np.cumsum(need) - need
    table = np.full((len(lens), max(1, int(need.max()))), -1, dtype=np.int32)
    inside = np.arange(table.shape[1])[None] < need[:, None]
    table[inside] = order[:total]
    return table, order, start


def _pools(case, blocks, gen, dtype):
    """K and V pools of a model's values: unit normals, keys with an offset for each channel and
    values with a scale for each token, quantised block by block."""
    hkv, block, d = case["kv_heads"], case["block"], case["head_dim"]
    k_pool = torch.empty(blocks, hkv, block, 9 * d // 16, dtype=torch.uint8, device=DEV)
    v_pool = torch.empty_like(k_pool)
    offset = _randn(gen, hkv, 1, d)
    step = max(1, (1 << 26) // (hkv * block * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        k = (_randn(gen, n, hkv, block, d) + offset).to(dtype)
        v = (_randn(gen, n, hkv, block, d) * (0.5 + _randn(gen, n, hkv, block, 1).abs())).to(dtype)
        k_pool[b:b + n] = _tile(*_quantise(k), False).view(n, hkv, block, -1)
        v_pool[b:b + n] = _tile(*_quantise(v), True).view(n, hkv, block, -1)
    return k_pool, v_pool


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, block = case["op"], case["block"]
    s = dict(case, type=TYPES[case["dtype"]] if "dtype" in case else None)
    if op == "attend":
        lens = _lengths(case)
        table, order, _ = _tables(lens, block, rng)
        s["k_pool"], s["v_pool"] = _pools(case, len(order), gen, s["type"])
        s["q"] = _randn(gen, case["seqs"], case["heads"], case["head_dim"]).to(s["type"])
        s["out"] = torch.empty_like(s["q"])
        s["tables"] = torch.from_numpy(table).to(DEV)
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        s["scale"] = 1.0 / math.sqrt(case["head_dim"])
        # the workspace that a serving loop holds: 256 + 16 bytes a row for the launch's order; of a
        # split call two words, the unnormalised row and a record for each partition
        rows = case["seqs"] * case["heads"]
        if case["partition"]:
            parts = _blocks(table.shape[1] * block, case["partition"])
            size = rows * (4 + parts * (24 + 4 * case["head_dim"])) + 2048
        else:
            size = 256 + 16 * rows if case["plan"] else 0
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
    elif op in ("store", "load"):
        t, hkv, d = case["tokens"], case["kv_heads"], case["head_dim"]
        blocks = max(1, math.ceil(1.25 * _blocks(t, block)))
        if op == "store" and case["scattered"]:  # each token in a block of another sequence
            blocks = max(blocks, t)
            slots = rng.permutation(blocks)[:t] * block + rng.integers(0, block, t)
        else:  # whole blocks in table order
            order = rng.permutation(blocks)[:_blocks(t, block)]
            slots = (order[:, None] * block + np.arange(block)[None]).reshape(-1)[:t]
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).to(DEV)
        if op == "load":
            s["k_pool"], s["v_pool"] = _pools(case, blocks, gen, s["type"])
        else:
            s["k_pool"] = torch.zeros(blocks, hkv, block, 9 * d // 16, dtype=torch.uint8, device=DEV)
            s["v_pool"] = torch.zeros_like(s["k_pool"])
            if case["fused"]:  # rows of a projection [queries | keys | values], one query head a KV head
                rows = _randn(gen, t, 3, hkv, d).to(s["type"])
                s["key"], s["value"] = rows[:, 1], rows[:, 2]
            else:
                s["key"] = _randn(gen, t, hkv, d).to(s["type"])
                s["value"] = _randn(gen, t, hkv, d).to(s["type"])
        s["key_out"] = torch.empty(t, hkv, d, dtype=s["type"], device=DEV)
        s["value_out"] = torch.empty_like(s["key_out"])
    else:
        new = _new_tokens(case)
        old = _lengths(case) if op == "extend" else np.zeros_like(new)
        after = old + new
        table, order, start = _tables(after, block, rng)
        had = _blocks(old, block)
        # the blocks that the requests hold already stay; the rest of the pool is the free stack
        rest = np.arange(table.shape[1])[None] >= had[:, None]
        held = set(table[~rest].tolist())
        free = np.array([b for b in order.tolist() if b not in held], dtype=np.int32)
        table[rest] = -1
        stack = np.full(len(order), -1, dtype=np.int32)
        stack[:len(free)] = free
        s["tables"] = torch.from_numpy(table).to(DEV)
        s["lens"] = torch.from_numpy(old.astype(np.int32)).to(DEV)
        s["new"] = torch.from_numpy(new.astype(np.int32)).to(DEV)
        s["free_list"] = torch.from_numpy(stack).to(DEV)
        s["free_count"] = torch.tensor([len(free)], dtype=torch.int32, device=DEV)
        s["lens_out"], s["count_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["free_count"])
        s["done"] = torch.ones_like(s["lens"])
        rows = int(new.sum()) + case.get("pad", 0)
        s["query_start"] = torch.empty(case["seqs"] + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(rows, dtype=torch.int64, device=DEV)
        s["positions"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["workspace"] = torch.empty(4 * case["seqs"] + 1024, dtype=torch.uint8, device=DEV)
    return s


# ---- the 4-bit format ----------------------------------------------------------------------

def _quantise(x):
    """Codes [..., D] (uint8) and (scale, minimum) [..., D / 64, 2] in x's type."""
    runs = x.float().unflatten(-1, (-1, RUN))
    least, most = runs.amin(-1), runs.amax(-1)
    scale = ((most - least) / 15.0).to(x.dtype)
    q = torch.floor((runs - least[..., None]) / scale.float()[..., None] + 0.5)
    q = torch.where(scale[..., None] > 0, q.clamp(0, 15), torch.zeros_like(q))
    return q.to(torch.uint8).flatten(-2), torch.stack([scale, least.to(x.dtype)], -1)


def _tile(codes, pairs, is_v):
    """Tiles [..., bytes] of codes [..., block, D] and pairs [..., block, D / 64, 2]."""
    lead, (block, d) = codes.shape[:-2], codes.shape[-2:]
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    if is_v:
        packed = packed.reshape(*lead, block // 2, 2, d // 4, 2).transpose(-3, -2)
    return torch.cat([packed.reshape(*lead, -1),
                      pairs.contiguous().view(torch.uint8).reshape(*lead, -1)], -1)


def _untile(tiles, block, d, dtype, is_v):
    """Values [..., block, D] in 32 bits of tiles [..., bytes]."""
    lead = tiles.shape[:-1]
    packed, pairs = tiles[..., :block * d // 2], tiles[..., block * d // 2:]
    if is_v:
        packed = packed.reshape(*lead, block // 2, d // 4, 2, 2).transpose(-3, -2)
    packed = packed.reshape(*lead, block, d // 2)
    codes = torch.stack([packed & 15, packed >> 4], -1).float()
    pairs = pairs.contiguous().view(dtype).reshape(*lead, block, d // RUN, 2).float()
    codes = codes.reshape(*lead, block, d // RUN, RUN)
    return (pairs[..., 1:] + codes * pairs[..., :1]).reshape(*lead, block, d)


def _places(slots, hkv, block, d, is_v):
    """Indices of the codes' bytes and of the pairs' bytes of slots [T] in [blocks][heads][tile]."""
    b, i = (slots // block)[:, None, None], slots % block
    head, byte = torch.arange(hkv, device=DEV)[None, :, None], torch.arange(d // 2, device=DEV)
    if is_v:
        byte = (i // 2 * d + i % 2 * 2)[:, None] + byte // 2 * 4 + byte % 2
    else:
        byte = (i * (d // 2))[:, None] + byte
    n = d // RUN * 4
    pair = (block * d // 2 + i * n)[:, None] + torch.arange(n, device=DEV)
    return (b, head, byte[:, None]), (b, head, pair[:, None])


# ---- plain forms ---------------------------------------------------------------------------

def _attend_plain(s):
    d, block, hkv = s["head_dim"], s["block"], s["kv_heads"]
    seqs, group = s["seqs"], s["heads"] // hkv
    at = s["tables"].clamp(min=0).long()

    def cached(pool, is_v):  # [S, heads, L, D]
        x = _untile(pool[at].flatten(3), block, d, s["type"], is_v)
        return x.transpose(1, 2).reshape(seqs, hkv, -1, d)

    q = s["q"].float().view(seqs, hkv, group, d)
    scores = torch.matmul(q, cached(s["k_pool"], False).transpose(-1, -2)) * s["scale"]
    unseen = torch.arange(scores.shape[-1], device=DEV) >= s["lens"][:, None]
    scores = scores.masked_fill(unseen[:, None, None], -math.inf)
    most = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(most > -math.inf, most, torch.zeros_like(most)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, cached(s["v_pool"], True)) / torch.where(total > 0, total, 1.0)
    return out.reshape(seqs, s["heads"], d).to(s["type"])


def _put(pool, x, slots, is_v):
    """Quantises the rows x [T, heads, D] into their slots."""
    codes, pairs = _quantise(x)
    at_codes, at_pairs = _places(slots, x.shape[1], pool.shape[2], x.shape[2], is_v)
    tiles = pool.view(pool.shape[0], pool.shape[1], -1)
    tiles[at_codes] = codes[..., 0::2] | (codes[..., 1::2] << 4)
    tiles[at_pairs] = pairs.contiguous().view(torch.uint8).flatten(-2)


def _get(pool, slots, d, dtype, is_v):
    """The rows [T, heads, D] that slots hold."""
    at_codes, at_pairs = _places(slots, pool.shape[1], pool.shape[2], d, is_v)
    tiles = pool.view(pool.shape[0], pool.shape[1], -1)
    packed, pairs = tiles[at_codes], tiles[at_pairs].view(dtype).float()
    codes = torch.stack([packed & 15, packed >> 4], -1).float().reshape(*packed.shape[:2], -1, RUN)
    pairs = pairs.reshape(*packed.shape[:2], -1, 2)
    return (pairs[..., 1:] + codes * pairs[..., :1]).flatten(-2).to(dtype)


def _extend_plain(s, lens_out, count_out):
    """Fills the tables' new entries, query_start, slots, positions, lengths and the free count."""
    block, table = s["block"], s["tables"]
    old, new = s["lens"].long(), s["new"].long()
    seqs, width = table.shape
    held, after = (old + block - 1) // block, (old + new + block - 1) // block
    need = after - held
    first = torch.cumsum(need, 0) - need
    column = torch.arange(width, device=DEV)
    fresh = (column >= held[:, None]) & (column < after[:, None])
    top = s["free_count"].long() - 1
    at = (top - first[:, None] - (column - held[:, None])).clamp(0, len(s["free_list"]) - 1)
    table.copy_(torch.where(fresh, s["free_list"][at], table))
    ends = torch.cumsum(new, 0)
    s["query_start"][:1] = 0
    s["query_start"][1:] = ends
    row = torch.arange(len(s["slots"]), device=DEV)
    real = row < ends[-1]
    seq = torch.searchsorted(ends, row, right=True).clamp(max=seqs - 1)
    pos = torch.where(real, old[seq] + row - (ends - new)[seq], 0)
    s["slots"].copy_(torch.where(real, table[seq, pos // block].long() * block + pos % block, -1))
    s["positions"].copy_(pos)
    lens_out.copy_(old + new)
    count_out.copy_(s["free_count"] - need.sum())


def _release_plain(s):
    """Pushes the blocks of the requests that are done, last request and last block first."""
    block, table = s["block"], s["tables"]
    held = torch.where(s["done"] != 0, (s["lens"].long() + block - 1) // block, 0)
    behind = held.sum() - torch.cumsum(held, 0)
    column = torch.arange(table.shape[1], device=DEV)
    gone = column < held[:, None]
    at = s["free_count"].long() + behind[:, None] + held[:, None] - 1 - column
    # an entry that is not pushed goes to a spare place behind the stack
    size = len(s["free_list"])
    stack = torch.cat([s["free_list"], s["free_list"][:1]])
    stack[torch.where(gone, at, size)] = table
    s["free_list"].copy_(stack[:size])
    table.masked_fill_(gone, -1)
    s["free_count"].add_(held.sum())
    s["lens"].mul_(s["done"] == 0)


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_312_gb300 as pkv
    if op == "attend":
        if not own:
            return _attend_plain(s)
        pkv.paged_decode_attention_q4(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"],
                                      s["lens"], s["scale"], s["block"], s["kv_heads"],
                                      partition_size=s["partition"], workspace=s["workspace"])
        return s["out"]
    if op in ("store", "load"):
        if not own:
            if op == "store":
                _put(s["k_pool"], s["key"], s["slots"], False)
                _put(s["v_pool"], s["value"], s["slots"], True)
            return [_get(s["k_pool"], s["slots"], s["head_dim"], s["type"], False),
                    _get(s["v_pool"], s["slots"], s["head_dim"], s["type"], True)]
        if op == "store":
            pkv.kv_write_q4(s["k_pool"], s["v_pool"], s["key"], s["value"], s["slots"])
        pkv.kv_read_q4(s["key_out"], s["value_out"], s["k_pool"], s["v_pool"], s["slots"])
        return [s["key_out"], s["value_out"]]
    lens_out, count_out = s["lens_out"], s["count_out"]
    if op == "turnover":  # lengths and count change in place, and come back with the release
        lens_out, count_out = s["lens"], s["free_count"]
    if own:
        pkv.tables_extend(s["tables"], s["lens"], s["new"], s["free_list"], s["free_count"],
                          s["block"], s["query_start"], s["slots"], s["positions"], s["workspace"],
                          lens_out=lens_out, free_count_out=count_out)
        if op == "turnover":
            pkv.tables_release(s["tables"], s["lens"], s["done"], s["free_list"], s["free_count"],
                               s["block"], s["workspace"])
    else:
        _extend_plain(s, lens_out, count_out)
        if op == "turnover":
            _release_plain(s)
    return {"tables": s["tables"], "lens": lens_out, "count": count_out, "free": s["free_list"],
            "query_start": s["query_start"], "slots": s["slots"], "positions": s["positions"]}


# ---- work and exact results ----------------------------------------------------------------

def work(case):
    if case["op"] == "attend":
        tokens, d = int(_lengths(case).sum()), case["head_dim"]
        q = case["seqs"] * case["heads"] * d * 2
        entries = int(_blocks(_lengths(case), case["block"]).sum()) + case["seqs"]
        return {"bytes": tokens * case["kv_heads"] * 2 * (9 * d // 16) + 2 * q + 4 * entries,
                "flops": 4 * tokens * case["heads"] * d}
    if case["op"] in ("store", "load"):
        n = 2 * case["tokens"] * case["kv_heads"] * case["head_dim"]  # elements of K and V
        store = case["op"] == "store"
        # rows read and tiles written; tiles read and rows written; the slots
        size = n * 2 + n * 9 // 16 + 8 * case["tokens"]
        return {"bytes": size * (2 if store else 1), "flops": n * (5 if store else 2)}
    new = _new_tokens(case)
    old = _lengths(case) if case["op"] == "extend" else np.zeros_like(new)
    need = int((_blocks(old + new, case["block"]) - _blocks(old, case["block"])).sum())
    rows = int(new.sum()) + case.get("pad", 0)
    size = 12 * rows + 8 * need + 16 * case["seqs"]
    if case["op"] == "turnover":
        size += 12 * need + 12 * case["seqs"]
    return {"bytes": size, "flops": 4 * rows}


def _values64(pool, at, block, d, dtype, is_v):
    """Values [blocks, block, D] in 64 bits of one head's tiles, taken apart byte by byte."""
    tiles = pool[at].flatten(1)
    i, e = torch.arange(block, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    byte = i // 2 * d + e // 4 * 4 + i % 2 * 2 + e % 4 // 2 if is_v else i * (d // 2) + e // 2
    code = (tiles[:, byte] >> (e % 2 * 4).to(torch.uint8)) & 15
    words = tiles[:, block * d // 2:].contiguous().view(dtype).double()
    pair = (i * (d // RUN) + e // RUN) * 2
    return words[:, pair + 1] + code.double() * words[:, pair]


def _exact_attend(case, s):
    lens = _lengths(case).tolist()
    d, block, hkv = case["head_dim"], case["block"], case["kv_heads"]
    group = case["heads"] // hkv
    if 4 * sum(lens) * case["heads"] * d > 2e11:
        return None
    out = torch.zeros(case["seqs"], case["heads"], d, dtype=torch.float64, device=DEV)
    for n, length in enumerate(lens):
        if not length:
            continue
        at = s["tables"][n, :_blocks(length, block)].long()
        for h in range(hkv):
            k, v = (_values64(s[pool][:, h], at, block, d, s["type"], is_v).reshape(-1, d)[:length]
                    for pool, is_v in (("k_pool", False), ("v_pool", True)))
            heads = slice(h * group, (h + 1) * group)
            p = torch.softmax((s["q"][n, heads].double() @ k.T) * s["scale"], -1)
            out[n, heads] = p @ v
    return out


def _quantised64(x):
    """What the rows x stand for once they are held in 4 bits, in 64 bits."""
    runs = x.double().unflatten(-1, (-1, RUN))
    least = runs.amin(-1, keepdim=True)
    scale = ((runs.amax(-1, keepdim=True) - least) / 15).to(x.dtype).double()
    codes = ((runs - least) / torch.where(scale > 0, scale, math.inf) + 0.5).floor().clamp(0, 15)
    return (least + codes * scale).flatten(-2)


def _exact_tables(case, s):
    """Request by request, block by block, on the host."""
    block, turnover = case["block"], case["op"] == "turnover"
    table, stack = s["tables"].cpu().numpy().copy(), s["free_list"].cpu().numpy().copy()
    lens, new = s["lens"].cpu().tolist(), s["new"].cpu().tolist()
    count, slots, positions, start = int(s["free_count"]), [], [], [0]
    for n, (old, more) in enumerate(zip(lens, new)):
        for p in range(_blocks(old, block), _blocks(old + more, block)):
            count -= 1
            table[n, p] = stack[count]
        p = np.arange(old, old + more)
        slots.append(table[n, p // block].astype(np.int64) * block + p % block)
        positions.append(p)
        start.append(start[-1] + more)
    after = [a + b for a, b in zip(lens, new)]
    if turnover:
        for n in reversed(range(len(after))):
            for p in reversed(range(_blocks(after[n], block))):
                stack[count] = table[n, p]
                table[n, p] = -1
                count += 1
        after = [0] * len(after)
    pad = case.get("pad", 0)
    return {"tables": table, "lens": np.array(after, np.int32), "count": np.array([count], np.int32),
            "free": stack, "query_start": np.array(start, np.int32),
            "slots": np.concatenate(slots + [np.full(pad, -1, np.int64)]),
            "positions": np.concatenate(positions + [np.zeros(pad)]).astype(np.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "store":
        return [_quantised64(s["key"]), _quantised64(s["value"])]
    if case["op"] == "load":
        d, block, slots = case["head_dim"], case["block"], s["slots"]
        blocks, inverse = torch.unique(slots // block, return_inverse=True)
        return [torch.stack([_values64(s[pool][:, h], blocks, block, d, s["type"], is_v)
                             [inverse, slots % block] for h in range(case["kv_heads"])], 1)
                for pool, is_v in (("k_pool", False), ("v_pool", True))]
    return _exact_tables(case, s)


if __name__ == "__main__":
    rng = random.Random(1)
    for c in listed() + [draw(rng) for _ in range(6)]:
        w = work(c)
        print("%-24s %12d bytes %14d flops" % (c.get("name", c["op"]), w["bytes"], w["flops"]))
