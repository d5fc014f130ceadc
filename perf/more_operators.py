"""Rotary positions and block-sparse decode attention: cases, plain forms, exact results.

Six kinds of case, one for each way in which a serving loop uses the operators:

rotate    rows of heads are rotated by their positions, on one axis or on several (a training
          step's or a re-positioned row's way back is the rotation the other way round)
append    new tokens' queries and keys are rotated, and keys and values stored in a paged cache
bounds    of the blocks that got new tokens: each channel's greatest and least key, in 8 bits
select    each sequence and KV head picks the blocks of its context that its query may attend to
          most, by an upper bound of the scores in them
attend    one query token per sequence attends over the picked blocks alone
sparse    bounds, select and attend of one decode step, one after the other

Rotation.  Pair i of a row's first rotary_dim elements turns by positions[axis of i] * inv_freq[i]
(radians); a pair is (i, i + rotary_dim / 2), or (2i, 2i + 1) where pairs are interleaved.  A
program keeps the frequencies as turns: round(2^64 * inv_freq / (2 pi)) modulo 2^64, as int64.

Bounds.  int8 [num_blocks][kv_heads][2][head_dim], greatest first, and a scale for each (block, KV
head), the least power of two 2^e, e >= -50, with every key of the block within 127 * 2^e.  The
greatest is rounded up, the least down: scale * bounds holds every key.  A block whose keys pass
127 * 2^50, or are not finite, has the scale infinity and bounds 0.

Select.  Of a context of n blocks that is longer than the K to be picked, the first and the most
recent ones are always kept, and the others of the greatest scores, the lowest block of equal
ones.  A query head is held in 8 bits as the keys are (rounded to nearest, halves up); a block's
score is the greatest of its KV head's query heads, of
    scale_q * scale * sum_d (q_d > 0 ? q_d * greatest_d : q_d * least_d),
a whole number times powers of two, exact in 32 bits.  A block that is kept whatever its score
has the score infinity.  The picked blocks come in ascending order as tiles block * kv_heads + kv_head
(-1 behind the last), with the number of tokens in them.
"""
import math
import random
from fractions import Fraction

import numpy as np
import torch

#: False: the plain forms below; True: the framework's kernels.
own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")


# ---- cases ---------------------------------------------------------------------------------

def _rotation(dtype, heads, head_dim, rotary, axes, interleaved, base, far):
    return dict(dtype=dtype, heads=heads, head_dim=head_dim, rotary=rotary, axes=axes,
                interleaved=interleaved, base=base, far=far)


def _context(dtype, heads, kv_heads, head_dim, block, seqs, lens, lo, hi):
    return dict(dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, block=block,
                seqs=seqs, lens=lens, lo=lo, hi=hi)


def listed():
    return [
        # the queries of four short chats on a small model: the call is all latency
        dict(_rotation("f16", 8, 64, 64, 1, True, 10000.0, 160), name="rotate-4", op="rotate",
             tokens=4, inverse=False),
        # the queries of a chunk of video frames: time, height and width
        dict(_rotation("bf16", 64, 128, 128, 3, False, 1e6, 4096), name="rotate-video-8192",
             op="rotate", tokens=8192, inverse=False),
        # the new tokens of one decode step of 64 sequences, rows of a fused projection
        dict(_rotation("bf16", 32, 128, 128, 1, False, 10000.0, 2048), name="append-step-64",
             op="append", kv_heads=32, block=16, tokens=64, pad=0, scattered=True, fused=True),
        # a padded batch of prompt chunks far into long documents
        dict(_rotation("bf16", 64, 128, 128, 1, False, 500000.0, 131072), name="append-chunks-8192",
             op="append", kv_heads=8, block=16, tokens=7777, pad=415, scattered=False, fused=True),
        # one decode step of a large grouped-query batch: a block a sequence
        dict(_context("bf16", 64, 8, 128, 16, 256, "lognormal", 16, 4096), name="bounds-step-256",
             op="bounds", new="one"),
        # a batch of prompts, every block of them
        dict(_context("bf16", 32, 32, 128, 16, 64, "uniform", 1, 2048), name="bounds-prompts-64",
             op="bounds", new="all"),
        # one request alone with a long document
        dict(_context("bf16", 64, 8, 128, 16, 1, "fixed", 131072, 131072), name="select-1x131072",
             op="select", picked=256),
        # a large batch of long contexts
        dict(_context("bf16", 64, 8, 128, 16, 64, "uniform", 1, 32768), name="select-64x32768",
             op="select", picked=128),
        # half of each context of a multi-head model's batch, no more
        dict(_context("bf16", 32, 32, 128, 16, 64, "uniform", 1, 2048), name="attend-mha32-64seq",
             op="attend", picked=32, partition=0, plan=False),
        # eight long contexts, 2048 tokens of each, split over the GPU
        dict(_context("bf16", 32, 8, 128, 32, 8, "fixed", 32768, 32768), name="attend-gqa32x8-8",
             op="attend", picked=64, partition=512, plan=False),
        # a decode step of four sequences of a small model
        dict(_context("f16", 8, 4, 64, 8, 4, "uniform", 1, 2048), name="sparse-4seq-d64",
             op="sparse", picked=32, partition=0, plan=False),
        # a decode step of 64 ragged contexts, at most 2048 tokens of each
        dict(_context("bf16", 64, 8, 128, 16, 64, "uniform", 1, 16384), name="sparse-gqa64x8-64seq",
             op="sparse", picked=128, partition=0, plan=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "bounds", "select", "select", "attend", "sparse"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("rotate", "append"):
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        rotary = rng.choice([head_dim, head_dim, 16 * rng.randint(1, head_dim // 16)])
        kv_heads, group = rng.randint(1, 8), rng.randint(1, 8)
        c = _rotation(dtype, kv_heads * group, head_dim, rotary, rng.choice([1, 1, 2, 3]),
                      rng.random() < 0.5, rng.choice([10000.0, 500000.0, 1e6]),
                      _spread(rng, 1, 1 << 20))
        tokens = _spread(rng, 1, min(32768, 20_000_000 // (c["heads"] * head_dim)))
        if op == "rotate":
            return dict(c, op=op, tokens=tokens, inverse=rng.random() < 0.5)
        return dict(c, op=op, kv_heads=kv_heads, block=rng.choice([8, 16, 32]), tokens=tokens,
                    pad=rng.choice([0, rng.randint(1, 500)]), scattered=rng.random() < 0.5,
                    fused=rng.random() < 0.5)
    kv_heads, group = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    seqs = _spread(rng, 1, 128)
    # at most a quarter of the largest listed case's cache rows in 16 bits
    hi = _spread(rng, 1, min(131072, 2_000_000 // (seqs * kv_heads)))
    c = _context(dtype, group * kv_heads, kv_heads, rng.choice([64, 128, 128]),
                 rng.choice([8, 16, 32]), seqs, rng.choice(["fixed", "uniform", "lognormal"]),
                 1, hi)
    if op == "bounds":
        return dict(c, op=op, new=rng.choice(["one", "some", "all"]))
    c["picked"] = _spread(rng, 2, 300)
    if op == "select":
        return dict(c, op=op)
    return dict(c, op=op, partition=rng.choice([0, 0, 1]) * 32 * rng.randint(4, 32),
                plan=rng.random() < 0.5)


def _blocks(n, block):
    return -(-n // block)


def _lengths(case):
    """The contexts' lengths: of the case alone, so that its work is known."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    rng = np.random.default_rng([n, lo, hi, case["block"]])
    if case["lens"] == "fixed":
        return np.full(n, hi, dtype=np.int64)
    if case["lens"] == "lognormal":
        x = np.exp(rng.normal(math.log(max(hi, 2)) - 2.0, 0.8, n))
        return np.clip(x, lo, hi).astype(np.int64)
    return rng.integers(lo, hi + 1, n)


def _new_tokens(case):
    """How many of each context's tokens are new, one at least."""
    lens = _lengths(case)
    if case.get("new", "one") == "one":
        return np.ones_like(lens)
    if case["new"] == "all":
        return lens
    return np.random.default_rng([case["seqs"], case["hi"]]).integers(1, lens + 1)


#: Blocks that are kept whatever their score: the first and the most recent one.
FIRST, RECENT = 1, 1


# ---- inputs --------------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _turns(inv_freq):
    """What a program keeps of the frequencies: turns a position, in units of 2^-64."""
    whole = [round(Fraction(f) * 2 ** 64 / TWO_PI) % 2 ** 64 for f in inv_freq]
    return torch.tensor([w - 2 ** 64 * (w >= 2 ** 63) for w in whole], dtype=torch.int64, device=DEV)


def _angles(case, rng, tokens):
    """Frequencies, the axis of each pair, and positions [tokens] or [axes, tokens]."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    inv_freq = [case["base"] ** (-i / pairs) for i in range(pairs)]
    s = {"inv_freq": torch.tensor(inv_freq, dtype=torch.float64, device=DEV),
         "turns": _turns(inv_freq), "pair_axis": None}
    start = rng.integers(0, case["far"])
    if axes == 1:  # tokens of several sequences, each in a row
        pos = (rng.integers(0, case["far"], 8)[:, None] + np.arange(_blocks(tokens, 8))).ravel()
        pos = pos[:tokens]
    else:  # frames of a grid, behind a text of a quarter of the tokens
        s["pair_axis"] = bytes(min(axes - 1, i * axes // pairs) for i in range(pairs))
        text = tokens // 4
        i, w = np.arange(tokens - text), 1 + int(math.sqrt(tokens)) // 4
        grid = [i // (w * w), i // w % w, i % w]
        pos = np.stack([np.concatenate([np.arange(text), text + grid[a]]) for a in range(axes)])
        pos = pos + start
    s["positions"] = torch.from_numpy(np.ascontiguousarray(pos, dtype=np.int32)).to(DEV)
    return s


def _tables(lens, block, rng):
    """Block tables over a shuffled pool a quarter larger than need be, -1 behind the last block."""
    need = _blocks(lens, block)
    total = int(need.sum())
    order = rng.permutation(max(1, math.ceil(1.25 * total))).astype(np.int32)
    table = np.full((len(lens), int(need.max())), -1, dtype=np.int32)
    table[np.arange(table.shape[1])[None] < need[:, None]] = order[:total]
    return torch.from_numpy(table).to(DEV), len(order)


def _keys(case, blocks, gen, dtype):
    """Blocks of keys as a model has them: an offset for each channel, a common part of a block's
    neighbouring tokens, and normals."""
    hkv, block, d = case["kv_heads"], case["block"], case["head_dim"]
    out = torch.empty(blocks, hkv, block, d, dtype=dtype, device=DEV)
    offset = _randn(gen, hkv, 1, d)
    for part in out.split(max(1, (1 << 26) // (hkv * block * d))):
        part.copy_(_randn(gen, *part.shape) + _randn(gen, len(part), hkv, 1, d) + offset)
    return out


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, dtype, d = case["op"], TYPES[case["dtype"]], case["head_dim"]
    s = dict(case, type=dtype)
    if op == "rotate":
        s.update(_angles(case, rng, case["tokens"]))
        s["x"] = _randn(gen, case["tokens"], case["heads"], d).to(dtype)
        s["out"] = torch.empty_like(s["x"])
        return s
    if op == "append":
        t, hkv, block = case["tokens"], case["kv_heads"], case["block"]
        rows = t + case["pad"]
        s.update(_angles(case, rng, rows))
        if case["fused"]:  # rows of one projection: queries, keys, values
            x = _randn(gen, rows, case["heads"] + 2 * hkv, d).to(dtype)
            s["q"], s["key"], s["value"] = x.split([case["heads"], hkv, hkv], 1)
        else:
            s["q"], s["key"], s["value"] = (_randn(gen, rows, h, d).to(dtype)
                                            for h in (case["heads"], hkv, hkv))
        blocks = max(1, math.ceil(1.25 * _blocks(t, block)))
        if case["scattered"]:  # each token in a block of another sequence
            blocks = t if t <= 1024 else blocks
            slots = rng.permutation(blocks * block)[:t]
        else:  # whole blocks in table order
            order = rng.permutation(blocks)[:_blocks(t, block)]
            slots = (order[:, None] * block + np.arange(block)[None]).reshape(-1)[:t]
        slots = np.concatenate([slots, np.full(case["pad"], -1)]).astype(np.int64)
        s["slots"] = torch.from_numpy(slots).to(DEV)
        s["k_cache"] = torch.zeros(blocks, hkv, block, d, dtype=dtype, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["q_out"] = torch.zeros(rows, case["heads"], d, dtype=dtype, device=DEV)
        return s
    lens, hkv = _lengths(case), case["kv_heads"]
    s["tables"], blocks = _tables(lens, case["block"], rng)
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
    keys = _keys(case, blocks, gen, dtype)
    s["bounds"] = torch.zeros(blocks, hkv, 2, d, dtype=torch.int8, device=DEV)
    s["scales"] = torch.zeros(blocks, hkv, device=DEV)
    if op in ("select", "sparse"):  # those of earlier steps
        for at in torch.arange(blocks, device=DEV).split(max(1, (1 << 26) // keys[0].numel())):
            s["bounds"][at], s["scales"][at] = _bounds_of(keys[at].float(), None)
    if op in ("bounds", "sparse"):
        new = _new_tokens(case)
        s["k_cache"], s["new"] = keys, torch.from_numpy(new.astype(np.int32)).to(DEV)
        s["max_new"] = int(new.max())
    if op == "bounds":
        return s
    s["q"] = _randn(gen, case["seqs"], case["heads"], d).to(dtype)
    s["picked_tiles"] = torch.full((case["seqs"], hkv, case["picked"]), -1, dtype=torch.int32,
                                   device=DEV)
    s["picked_lens"] = torch.zeros(case["seqs"], hkv, dtype=torch.int32, device=DEV)
    s["scores"] = torch.zeros(case["seqs"], hkv, s["tables"].shape[1], device=DEV)
    if op == "select":
        return s
    s["k_cache"] = keys
    s["v_cache"] = torch.empty_like(keys)
    for part in s["v_cache"].split(max(1, (1 << 26) // keys[0].numel())):
        part.copy_(_randn(gen, *part.shape))
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "attend":
        score = torch.rand(s["scores"].shape, generator=gen, device=DEV)
        _pick(s, score, s["picked_tiles"], s["picked_lens"])
    # the workspace that a serving loop holds: 256 + 16 bytes a row for the launch's order; of a
    # split call two words, the unnormalised row and a record for each partition
    rows = case["seqs"] * case["heads"]
    if case["partition"]:
        parts = _blocks(case["picked"] * case["block"], case["partition"])
        size = rows * (4 + parts * (24 + 4 * d)) + 2048
    else:
        size = 256 + 16 * rows if case["plan"] else 0
    s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
    return s


# ---- plain forms ---------------------------------------------------------------------------

def _rotated(s, x, sign=1.0):
    """The rows x [T, H, D] rotated, in 32 bits (the angles in 64)."""
    pos, r = s["positions"].double(), s["rotary"]
    if s["axes"] > 1:
        pos = pos[torch.tensor(list(s["pair_axis"]), device=DEV)].T
    else:
        pos = pos[:, None]
    angle = pos * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], (sign * angle.sin()).float()[:, None]
    x = x.float()
    rot = x[..., :r].unflatten(-1, (-1, 2) if s["interleaved"] else (2, -1))
    dim = -1 if s["interleaved"] else -2
    a, b = rot.unbind(dim)
    rot = torch.stack([a * cos - b * sin, b * cos + a * sin], dim).flatten(-2)
    return torch.cat([rot, x[..., r:]], -1)


def _append_plain(s):
    t, block = s["tokens"], s["block"]
    s["q_out"][:t] = _rotated(s, s["q"])[:t].to(s["type"])
    at, offset = s["slots"][:t] // block, s["slots"][:t] % block
    s["k_cache"][at, :, offset] = _rotated(s, s["key"])[:t].to(s["type"])
    s["v_cache"][at, :, offset] = s["value"][:t]


def _power(most):
    """The least 2^e, e >= -50, with most <= 127 * 2^e; infinity past e = 50."""
    f, e = torch.frexp(most)
    e = torch.where(f <= 127 / 128, e - 7, e - 6).clamp(-50, 51)
    e = torch.where(most > 0, e, -50)
    scale = ((e + 127) << 23).to(torch.int32).view(torch.float32)  # 2^e
    return torch.where((most < math.inf) & (e <= 50), scale, math.inf)


def _bounds_of(keys, seen):
    """Bounds and scales of blocks of keys [..., B, D] in 32 bits; seen [..., B, 1] or None."""
    most, least = keys, keys
    if seen is not None:
        most, least = keys.masked_fill(~seen, -math.inf), keys.masked_fill(~seen, math.inf)
    most, least = most.amax(-2), least.amin(-2)
    scale = _power(torch.maximum(most.abs(), least.abs()).amax(-1))
    most, least = torch.ceil(most / scale[..., None]), torch.floor(least / scale[..., None])
    both = torch.stack([most, least], -2)
    return torch.where(scale[..., None, None] < math.inf, both, 0.0).to(torch.int8), scale


def _bounds_plain(s):
    block, lens, new = s["block"], s["lens"].long(), s["new"].long()
    first, last = (lens - new) // block, (lens - 1) // block
    # column past a sequence's last block: that block again
    column = first[:, None] + torch.arange(_blocks(s["max_new"], block) + 1, device=DEV)
    column = torch.minimum(column, last[:, None])
    at = torch.gather(s["tables"].long(), 1, column)
    token = column[..., None] * block + torch.arange(block, device=DEV)
    seen = (token < lens[:, None, None])[:, :, None, :, None]
    s["bounds"][at], s["scales"][at] = _bounds_of(s["k_cache"][at].float(), seen)


def _descending(x):
    """The order of the last dimension from the greatest value, the lowest index of equal ones."""
    return torch.sort(x, dim=-1, descending=True, stable=True).indices


def _pick(s, score, tiles, lens):
    """The blocks of the greatest scores, the lowest of equal ones: tiles [S, heads, K] and their
    tokens [S, heads]."""
    block, hkv, k = s["block"], s["kv_heads"], s["picked"]
    n = (s["lens"].long() + block - 1) // block
    width = score.shape[-1]
    column = torch.arange(width, device=DEV)
    kept = (column < FIRST) | (column >= n[:, None] - RECENT)
    rank = torch.where(kept[:, None], 1, 0) * 2.0 + torch.where(score == math.inf, 1, 0)
    # by rank, then by score, both descending; stable, so the lowest block first
    order = _descending(score.masked_fill(score == math.inf, 0.0))
    real = (column < n[:, None])[:, None].expand_as(score)
    rank = torch.where(real, rank, -1.0)
    order = torch.gather(order, -1, _descending(torch.gather(rank, -1, order)))
    picked = order[..., :k]
    if width < k:
        picked = torch.cat([picked, picked.new_full((*picked.shape[:-1], k - width), width)], -1)
    count = n.clamp(max=k)[:, None, None]
    inside = torch.arange(k, device=DEV) < count
    picked = picked.masked_fill(~inside, 1 << 40).sort(-1).values
    at = picked.clamp(max=width - 1).flatten(1)
    head = torch.arange(hkv, device=DEV)[:, None]
    found = torch.gather(s["tables"].long(), 1, at).view_as(picked) * hkv + head
    tiles.copy_(torch.where(inside, found, -1))
    # whole blocks but for the context's last one, which is always among them
    lens.copy_((count * block - (n * block - s["lens"])[:, None, None])[..., 0].expand_as(lens))


def _select_plain(s):
    seqs, hkv, d, k = s["seqs"], s["kv_heads"], s["head_dim"], s["picked"]
    q = s["q"].float().view(seqs, hkv, -1, d)
    scale_q = _power(q.abs().amax(-1))
    q = torch.floor(q / scale_q[..., None] + 0.5)
    at = s["tables"].long().clamp(min=0)
    bounds = s["bounds"][at].float().transpose(1, 2)  # [S, heads, n, 2, D]
    both = torch.cat([q.clamp(min=0), q.clamp(max=0)], -1)  # whole numbers: sums are exact
    dots = torch.matmul(both, bounds.flatten(-2).transpose(-1, -2))
    scale = s["scales"][at].transpose(1, 2)
    score = (dots * scale_q[..., None]).amax(-2) * torch.where(scale < math.inf, scale, 1.0)
    score = score.masked_fill(scale == math.inf, math.inf)
    n = ((s["lens"].long() + s["block"] - 1) // s["block"])[:, None]
    column = torch.arange(score.shape[-1], device=DEV)
    kept = (column < FIRST) | (column >= n - RECENT) | (n <= k)
    score = score.masked_fill(kept[:, None], math.inf)
    s["scores"].copy_(torch.where((column < n)[:, None], score, s["scores"]))
    _pick(s, score, s["picked_tiles"], s["picked_lens"])


def _attend_plain(s):
    d, block, hkv, k = s["head_dim"], s["block"], s["kv_heads"], s["picked"]
    seqs = s["seqs"]
    at = s["picked_tiles"].long().clamp(min=0)
    keys, values = (s[c].view(-1, block, d)[at].float().reshape(seqs, hkv, k * block, d)
                    for c in ("k_cache", "v_cache"))
    q = s["q"].float().view(seqs, hkv, -1, d)
    scores = torch.matmul(q, keys.transpose(-1, -2)) * s["scale"]
    unseen = torch.arange(k * block, device=DEV) >= s["picked_lens"][..., None]
    scores = scores.masked_fill(unseen[:, :, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    out = torch.matmul(p, values) / p.sum(-1, keepdim=True)
    return out.reshape(seqs, s["heads"], d).to(s["type"])


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_312_gb300 as pkv
    if op == "rotate":
        if not own:
            return _rotated(s, s["x"], -1.0 if s["inverse"] else 1.0).to(s["type"])
        pkv.rope(s["out"], s["x"], s["positions"], s["turns"], pair_axis=s["pair_axis"],
                 interleaved=s["interleaved"], inverse=s["inverse"])
        return s["out"]
    if op == "append":
        if own:
            pkv.rope_write(s["q_out"], s["k_cache"], s["v_cache"], s["q"], s["key"], s["value"],
                           s["positions"], s["turns"], s["slots"], pair_axis=s["pair_axis"],
                           interleaved=s["interleaved"])
        else:
            _append_plain(s)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    got = {}
    if op in ("bounds", "sparse"):
        if own:
            pkv.block_bounds(s["bounds"], s["scales"], s["k_cache"], s["tables"], s["lens"],
                             s["new"], s["max_new"])
        else:
            _bounds_plain(s)
        got.update(bounds=s["bounds"], scales=s["scales"])
    if op in ("select", "sparse"):
        if own:
            pkv.select_blocks(s["picked_tiles"], s["picked_lens"], s["scores"], s["q"], s["bounds"],
                              s["scales"], s["tables"], s["lens"], s["block"], first_blocks=FIRST,
                              recent_blocks=RECENT)
        else:
            _select_plain(s)
        got.update(tiles=s["picked_tiles"], lens=s["picked_lens"], scores=s["scores"])
    if op in ("attend", "sparse"):
        if own:
            pkv.paged_decode_attention_selected(
                s["out"], s["q"], s["k_cache"], s["v_cache"], s["picked_tiles"], s["picked_lens"],
                s["scale"], s["block"], s["kv_heads"], partition_size=s["partition"],
                workspace=s["workspace"])
            got["out"] = s["out"]
        else:
            got["out"] = _attend_plain(s)
    return got


# ---- work and exact results ----------------------------------------------------------------

def work(case):
    size, d = 4 if case["dtype"] == "f32" else 2, case["head_dim"]
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * d * size + 4 * case["tokens"] * case["axes"] + 4 * case["rotary"],
                "flops": 3 * n * case["rotary"]}
    if case["op"] == "append":
        t, rows = case["tokens"], case["tokens"] + case["pad"]
        heads = case["heads"] + 2 * case["kv_heads"]
        return {"bytes": 2 * t * heads * d * size + rows * (8 + 4 * case["axes"]),
                "flops": 3 * t * (heads - case["kv_heads"]) * case["rotary"]}
    lens, block, hkv = _lengths(case), case["block"], case["kv_heads"]
    n, total, flops = _blocks(lens, block), 0, 0
    if case["op"] in ("bounds", "sparse"):
        first = (lens - _new_tokens(case)) // block
        keys = int((lens - first * block).sum()) * hkv * d
        total += keys * size + int((n - first).sum()) * (hkv * (2 * d + 4) + 4)
        flops += 2 * keys
    q = case["seqs"] * case["heads"] * d * size
    chosen = np.minimum(n, case.get("picked", 0))
    if case["op"] in ("select", "sparse"):
        scored = int(np.where(n > case["picked"], n - FIRST - RECENT, 0).sum()) * hkv
        # bounds read, scores written, the picked blocks' table entries read and tiles written
        total += scored * (2 * d + 4) + 4 * int(n.sum()) * hkv + 8 * int(chosen.sum()) * hkv + q
        flops += 2 * scored * (case["heads"] // hkv) * 2 * d
    if case["op"] in ("attend", "sparse"):
        tokens = int(np.minimum(lens, chosen * block).sum())
        total += tokens * hkv * 2 * d * size + 2 * q + 4 * int(chosen.sum()) * hkv
        flops += 4 * tokens * case["heads"] * d
    return {"bytes": total, "flops": flops}


def _turned(case, s, x, sign=1.0):
    """Rows rotated in 64 bits, as complex numbers."""
    half = case["rotary"] // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    pos = s["positions"].double().reshape(case["axes"], -1)
    axis = list(s["pair_axis"]) if s["pair_axis"] else [0] * half
    angle = torch.stack([pos[a] * f for a, f in zip(axis, s["inv_freq"])], -1)
    z = torch.complex(x[..., first].double(), x[..., second].double())
    z = z * torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    out = x.double()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exponent(most):
    """e of the scale of values up to most: 51 stands for infinity."""
    if not most < 127 * 2.0 ** 50 * (1 + 2.0 ** -30):
        return 51
    e = -50
    while most > 127 * 2.0 ** e:
        e += 1
    return e


def _exact_bounds(case, s):
    """Block by block; every (block, head) of one at once."""
    block, lens, new = case["block"], _lengths(case).tolist(), _new_tokens(case).tolist()
    bounds, scales = s["bounds"].clone(), s["scales"].clone()
    units = torch.tensor([2.0 ** e for e in range(-50, 51)] + [math.inf], dtype=torch.float64,
                         device=DEV)
    for n, (length, more) in enumerate(zip(lens, new)):
        first = (length - more) // block
        at = s["tables"][n, first:_blocks(length, block)].long()
        keys = s["k_cache"][at].double()
        tail = length - (_blocks(length, block) - 1) * block
        hi, lo = keys.amax(2), keys.amin(2)
        hi[-1], lo[-1] = keys[-1, :, :tail].amax(1), keys[-1, :, :tail].amin(1)
        most = torch.maximum(hi.abs().amax(-1), lo.abs().amax(-1))
        unit = units[torch.searchsorted(127 * units, most)]  # the first that is not less
        both = torch.stack([(hi / unit[..., None]).ceil(), (lo / unit[..., None]).floor()], 2)
        bounds[at] = both.masked_fill((unit == math.inf)[..., None, None], 0).to(torch.int8)
        scales[at] = unit.float()
    return bounds, scales


def _exact_select(case, s, bounds, scales):
    """Sequence by sequence and head by head, scores as whole numbers times powers of two."""
    lens, block, k = _lengths(case).tolist(), case["block"], case["picked"]
    hkv, d = case["kv_heads"], case["head_dim"]
    group = case["heads"] // hkv
    tiles = np.full((case["seqs"], hkv, k), -1, np.int32)
    scores, count = s["scores"].double(), np.zeros((case["seqs"], hkv), np.int32)
    q = s["q"].double()
    for i, length in enumerate(lens):
        n = _blocks(length, block)
        ids = s["tables"][i, :n].long()
        on_host = ids.cpu().numpy()
        scores[i, :, :n] = math.inf
        most = q[i].abs().amax(-1).cpu().tolist()
        for h in range(hkv):
            keep = np.arange(n)
            if n > k:
                rows = []
                for g in range(h * group, (h + 1) * group):
                    unit = 2.0 ** _exponent(most[g])
                    whole = torch.floor(q[i, g] / unit + 0.5)
                    up, down = bounds[ids, h].double().unbind(1)
                    rows.append(torch.where(whole > 0, whole * up, whole * down).sum(-1) * unit)
                row = torch.stack(rows).amax(0) * scales[ids, h].double()
                row = torch.where(scales[ids, h] == math.inf, math.inf, row)
                row[:FIRST] = math.inf
                row[n - RECENT:] = math.inf
                scores[i, h, :n] = row
                row = row.cpu().numpy().copy()
                always = np.zeros(n)
                always[:FIRST], always[n - RECENT:] = 1, 1
                keep = np.sort(np.lexsort((np.arange(n), -row, -always))[:k])
            tiles[i, h, :len(keep)] = on_host[keep] * hkv + h
            count[i, h] = sum(min(block, length - b * block) for b in keep.tolist())
    return torch.from_numpy(tiles), torch.from_numpy(count), scores


def _exact_attend(case, s, tiles, lens):
    d, block, hkv = case["head_dim"], case["block"], case["kv_heads"]
    group = case["heads"] // hkv
    keys, values = s["k_cache"].view(-1, block, d), s["v_cache"].view(-1, block, d)
    out = torch.zeros(case["seqs"], case["heads"], d, dtype=torch.float64, device=DEV)
    lens, tiles = lens.cpu().tolist(), tiles.to(DEV).long()
    for i in range(case["seqs"]):
        for h in range(hkv):
            length = lens[i][h]
            at = tiles[i, h, :_blocks(length, block)]
            k, v = (c[at].double().reshape(-1, d)[:length] for c in (keys, values))
            heads = slice(h * group, (h + 1) * group)
            out[i, heads] = torch.softmax((s["q"][i, heads].double() @ k.T) * s["scale"], -1) @ v
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rotate":
        return _turned(case, s, s["x"], -1.0 if case["inverse"] else 1.0)
    if op == "append":
        t, block = case["tokens"], case["block"]
        q, k, v = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
        q[:t] = _turned(case, s, s["q"])[:t]
        at, offset = s["slots"][:t] // block, s["slots"][:t] % block
        k[at, :, offset], v[at, :, offset] = _turned(case, s, s["key"])[:t], s["value"][:t].double()
        return {"q": q, "k_cache": k, "v_cache": v}
    got = {}
    bounds, scales = s["bounds"], s["scales"]
    if op in ("bounds", "sparse"):
        bounds, scales = _exact_bounds(case, s)
        got.update(bounds=bounds, scales=scales.double())
    if op in ("select", "sparse"):
        if case["seqs"] * case["heads"] > 10000:
            return None
        tiles, lens, scores = _exact_select(case, s, bounds, scales)
        got.update(tiles=tiles, lens=lens, scores=scores)
    if op in ("attend", "sparse"):
        if op == "attend":
            tiles, lens = s["picked_tiles"], s["picked_lens"]
        got["out"] = _exact_attend(case, s, tiles, lens)
    return got


if __name__ == "__main__":
    rng = random.Random(1)
    for c in listed() + [draw(rng) for _ in range(6)]:
        w = work(c)
        print("%-24s %12d bytes %14d flops" % (c.get("name", c["op"]), w["bytes"], w["flops"]))
