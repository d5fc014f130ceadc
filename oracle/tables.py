"""Oracle of the block tables built on the GPU: requests one by one, blocks one
by one, on Python lists."""
from __future__ import annotations


def extend(tables, lens, new, stack, count, block, num_blocks, max_tokens):
    """One step of a batch.  tables: list of lists (changed in place); stack:
    list of ids.  Returns (lens, count, query_start, slots, positions, refused,
    bad lengths)."""
    width = len(tables[0]) if tables else 0
    asked, bad = [], False
    for n, (old, more) in enumerate(zip(lens, new)):
        fits = old >= 0 and more >= 0 and old + more <= width * block
        bad = bad or not fits
        asked.append(more if fits else 0)
    need = [-(-(old + a) // block) + (-old // block) if a else 0 for old, a in zip(lens, asked)]
    refused = not 0 <= count <= num_blocks or sum(need) > count or sum(asked) > max_tokens
    start = [0]
    if refused:
        return list(lens), count, [0] * (len(lens) + 1), [-1] * max_tokens, [0] * max_tokens, True, bad
    slots, positions, after = [], [], []
    for n, (old, more) in enumerate(zip(lens, asked)):
        for p in range(old, old + more):
            if p % block == 0:
                count -= 1
                tables[n][p // block] = stack[count]
            entry = tables[n][p // block]
            slots.append(entry * block + p % block if 0 <= entry < num_blocks else -1)
            positions.append(p)
        after.append(old + more)
        start.append(start[-1] + more)
    pad = max_tokens - len(slots)
    return after, count, start, slots + [-1] * pad, positions + [0] * pad, False, bad


def release(tables, lens, done, stack, count, block, num_blocks):
    """Gives the blocks of finished requests back, last request and last block
    first; everything in place.  Returns (count, refused, bad lengths)."""
    width = len(tables[0]) if tables else 0
    held, bad = [], False
    for old, d in zip(lens, done):
        fits = 0 <= old <= width * block
        bad = bad or (bool(d) and not fits)
        held.append(-(-old // block) if d and fits else 0)
    if count < 0 or count + sum(held) > num_blocks:
        return count, True, bad
    for n in reversed(range(len(lens))):
        for j in reversed(range(held[n])):
            stack[count] = tables[n][j]
            tables[n][j] = -1
            count += 1
        if held[n]:
            lens[n] = 0
    return count, False, bad
