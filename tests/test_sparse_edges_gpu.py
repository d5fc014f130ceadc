"""GPU: calls of the operators over selected blocks, and of the rotations, that their documents
allow and that ordinary use seldom makes, against the oracle."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import sparse as oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


class Selection:
    """One selection's arguments and outputs: random bounds and queries, blocks that repeat."""

    def __init__(self, group, d, width, k, seed, S=3, hkv=2, nb=300, block=8):
        g = torch.Generator().manual_seed(seed)
        hi = torch.randint(-40, 128, (nb, hkv, d), generator=g)
        lo = (hi - torch.randint(0, 90, (nb, hkv, d), generator=g)).clamp(min=-127)
        self.bounds = torch.stack([hi, lo], 2).to(torch.int8)
        self.scales = 2.0 ** torch.randint(-7, -2, (nb, hkv), generator=g).float()
        self.table = torch.randint(0, nb, (S, width), generator=g, dtype=torch.int32)
        self.q = torch.randn(S, group * hkv, d, generator=g).bfloat16()
        self.lens = [width * block, width * block // 2 + 1, 3]
        self.block, self.k = block, k
        self.sel, self.n = i32(np.zeros((S, hkv, k))), i32(np.zeros((S, hkv)))
        self.scores = torch.zeros(S, hkv, width, device=DEV)
        self.args = [self.sel, self.n, self.scores, self.q.to(DEV), self.bounds.to(DEV),
                     self.scales.to(DEV), self.table.to(DEV), i32(self.lens), block]

    def run(self, stream=None):
        pkv.select_blocks(*self.args, stream=stream)

    def check(self):
        want = oracle.select(self.q.double().numpy(), self.bounds.numpy(),
                             self.scales.double().numpy(), self.table.tolist(), self.lens,
                             self.block, self.k)
        assert (self.sel.cpu().numpy() == want[0]).all()
        assert (self.n.cpu().numpy() == want[1]).all()
        assert (self.scores.cpu().double().numpy() == want[2]).all()


def test_threads_may_select_with_other_numbers_of_query_heads():
    """Four threads with streams of their own, whose launches of the same kernels need other sizes
    of shared memory (past the 48 KB that every launch may have)."""
    sets = [[Selection(group, 128, width, 20, 7 * i + j)
             for j, (group, width) in enumerate(((a, 500), (b, 40), (a, 40), (b, 700)))]
            for i, (a, b) in enumerate(((32, 128), (128, 30), (64, 28), (100, 128)))]
    torch.cuda.synchronize()
    errors = []

    def work(mine):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                for s in mine:
                    s.run(stream)
            stream.synchronize()
        except Exception as e:  # shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(mine,)) for mine in sets]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    assert pkv.device_status() == 0
    for mine in sets:
        for s in mine:
            s.check()


@pytest.mark.parametrize("width", [60, 520, 1500, 2100, 9000])
@pytest.mark.parametrize("zeros", [[0.0], [-0.0], [0.0, -0.0]])
def test_scales_of_zero_give_equal_scores(zeros, width):
    """Pools whose scales start at zero, over bounds of any bytes: sums of both signs times zero
    are equal scores, of which the lowest blocks are picked."""
    s = Selection(4, 64, width, 25, width)
    s.scales[::2, 0] = torch.tensor(zeros)[torch.arange(150) % len(zeros)]
    s.scales[:, 1] = torch.tensor(zeros)[torch.arange(300) % len(zeros)]
    s.bounds[::3] = -s.bounds[::3]
    s.args[4], s.args[5] = s.bounds.to(DEV), s.scales.to(DEV)
    s.run()
    assert pkv.device_status() == 0
    s.check()


@pytest.mark.parametrize("form", [list, np.array, lambda a: np.array(a, dtype=np.int32),
                                  torch.tensor, bytearray])
def test_the_axes_of_pairs_in_any_form(form):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 3, 64, generator=g).bfloat16().to(DEV)
    pos = i32(torch.randint(0, 1000, (3, 9), generator=g))
    turns = pkv.rope_turns([10000.0 ** (-i / 32) for i in range(32)], DEV)
    axes = [i * 3 // 32 for i in range(32)]
    want, got = torch.empty_like(x), torch.empty_like(x)
    pkv.rope(want, x, pos, turns, pair_axis=bytes(axes))
    pkv.rope(got, x, pos, turns, pair_axis=form(axes))
    assert torch.equal(want, got)
    with pytest.raises(ValueError):
        pkv.rope(got, x, pos, turns, pair_axis=32)
    with pytest.raises(ValueError):  # the right number of bytes, of eight numbers
        pkv.rope(got, x, pos, turns, pair_axis=np.array(axes[:8], dtype=np.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,d,block,partition", [
    (8, 128, 16, 64), (1, 64, 8, 64), (5, 64, 32, 32), (7, 128, 32, 256),  # clusters
    (12, 128, 16, 64),                                                     # a plan
    (8, 128, 16, 0), (3, 64, 8, 0), (16, 64, 32, 0)])                      # unsplit
def test_weights_are_held_in_more_than_16_bits(dtype, group, d, block, partition):
    """Three tokens of each context count, side by side: the first one's weight is 1, the others'
    are numbers that one rounding to 16 bits would leave up to 2^-9 (bf16) or 2^-12 (fp16) off.
    All else is exact: head h's query is 1 in channel h and 0 elsewhere, so that a key's channel h
    is its score (0; sixty-fourths down to -1.5; -240, whose weight is 0), values are 1 or -1.

    A weight's relative error: its score in base 2, at most 2.2, rounded twice (log2 e and the
    product), 2 * 2.2 * 2^-24 * ln 2; 2^x 2^-22; together below 2^-21.  A sum of three weights, a
    rescale by 2^x of each of the two joins, a few roundings: below 2^-19 for the weighted values
    and for the weights each.  The two-part weight itself: half a step of half a step, 2^-16 in
    bf16; 2^-22 in fp16, or half of its least step, 2^-25, against weights of 0.22 and more.
    With values of 1 and -1 the output is off by at most 2 * 2^-19 and that: below 2^-15 and
    2^-17."""
    S, hkv, k = 4, 2, 40
    nb = S * k
    g = torch.Generator().manual_seed(group * d)
    tokens = k * block
    kd = torch.zeros(S, hkv, tokens, d)
    kd[..., :group] = -240.0
    vd = torch.randint(0, 2, (S, hkv, tokens, d), generator=g) * 2.0 - 1.0
    lens = torch.randint(9, tokens + 1, (S, hkv), generator=g, dtype=torch.int32)
    lens[0] = tokens
    for s in range(S):
        for h in range(hkv):
            at = int(torch.randint(0, int(lens[s, h]) // 8, (1,), generator=g)) * 8
            kd[s, h, at, :group] = 0.0
            kd[s, h, at + 1:at + 3, :group] = -torch.randint(1, 97, (2, group), generator=g) / 64.0
    # whole contexts into a shuffled pool
    order = torch.randperm(nb, generator=g).view(S, k)
    kc, vc = (torch.empty(nb, hkv, block, d) for _ in range(2))
    for pool, x in ((kc, kd), (vc, vd)):
        pool[order] = x.view(S, hkv, k, block, d).transpose(1, 2)
    tiles = (order[:, None] * hkv + torch.arange(hkv)[None, :, None]).to(torch.int32)
    q = torch.eye(d)[:group].repeat(S, hkv, 1)
    ws = torch.empty(pkv.decode_workspace_bytes(S, group * hkv, d, tokens, partition),
                     dtype=torch.uint8, device=DEV) if partition else None
    out = torch.full((S, group * hkv, d), 9.0, device=DEV)
    pkv.paged_decode_attention_selected(out, *(x.to(dtype).to(DEV) for x in (q, kc, vc)),
                                        i32(tiles), lens.to(DEV), 1.0, block, hkv, partition, ws)
    assert pkv.device_status() == 0
    # the same with weights as they are, and rounded once
    want, once = np.zeros((2, S, hkv, group, d))
    for s in range(S):
        for h in range(hkv):
            n = int(lens[s, h])
            w = np.exp(kd[s, h, :n, :group].double().numpy()).T
            rounded = torch.from_numpy(w).to(dtype).double().numpy()
            v = vd[s, h, :n].double().numpy()
            want[s, h] = w @ v / w.sum(-1, keepdims=True)
            once[s, h] = rounded @ v / w.sum(-1, keepdims=True)
    bound = 2.0 ** (-15 if dtype is torch.bfloat16 else -17)
    assert np.abs(once - want).max() > 2 * bound  # the bound tells them apart
    off = np.abs(out.cpu().double().numpy().reshape(want.shape) - want).max()
    assert off <= bound, off


@pytest.mark.parametrize("dtype,partition", [("bf16", 0), ("f16", 64)])
def test_bounds_and_selection_over_a_4_bit_cache(dtype, partition):
    """Bounds of a 4-bit cache's keys, as its document says: the blocks' rows are read back, a
    cache of blocks that are a sequence each; their bounds go to the blocks' places.  They hold
    the keys that the pool stands for but for the rounding of the rows; the selection by them and
    the attention over it, each against its oracle."""
    from test_q4_attention_gpu import DT, Case, check, codes_of
    hq, hkv, d, block, k = 8, 2, 128, 16, 6
    case = Case(DT[dtype], hq, hkv, d, block, [500, 95, 0, 301, 1, 97])
    S, width = case.tables.shape
    nb = case.k.shape[0]
    kp, vp = case.k.to(DEV), case.v.to(DEV)
    ids, held = [], []  # blocks, and the tokens in each
    for row, n in zip(case.tables.tolist(), case.lens.tolist()):
        for j in range(-(-n // block)):
            ids.append(row[j])
            held.append(min(block, n - j * block))
    n = len(ids)
    at = torch.tensor(ids, device=DEV)
    slots = (at[:, None] * block + torch.arange(block, device=DEV)).flatten()
    key, value = (torch.empty(n * block, hkv, d, dtype=DT[dtype], device=DEV) for _ in range(2))
    pkv.kv_read_q4(key, value, kp, vp, slots)
    rows = key.view(n, block, hkv, d).transpose(1, 2).contiguous()
    some, some_scales = (torch.empty(n, hkv, 2, d, dtype=torch.int8, device=DEV),
                         torch.empty(n, hkv, device=DEV))
    pkv.block_bounds(some, some_scales, rows, torch.arange(n, device=DEV).int()[:, None], i32(held),
                     i32(held), block)
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device=DEV)
    scales = torch.zeros(nb, hkv, device=DEV)
    bounds[at], scales[at] = some, some_scales
    sel, slens = i32(np.zeros((S, hkv, k))), i32(np.zeros((S, hkv)))
    scores = torch.zeros(S, hkv, width, device=DEV)
    pkv.select_blocks(sel, slens, scores, case.q.to(DEV), bounds, scales, case.tables.to(DEV),
                      case.lens.to(DEV), block)
    ws = torch.empty(pkv.decode_workspace_bytes(S, hq, d, k * block, partition), dtype=torch.uint8,
                     device=DEV) if partition else None
    out = torch.empty(S, hq, d, device=DEV)
    pkv.paged_decode_attention_selected(out, case.q.to(DEV), kp, vp, sel, slens, case.scale, block,
                                        hkv, partition, ws)
    # bounds: the oracle's of the rows, around the keys
    hb, hsc = np.zeros((n, hkv, 2, d), np.int8), np.zeros((n, hkv))
    assert oracle.block_bounds(hb, hsc, rows.cpu().double().numpy(), [[i] for i in range(n)], held,
                               held, block) == 0
    assert (some.cpu().numpy() == hb).all() and (some_scales.cpu().numpy() == hsc).all()
    codes, s, m = codes_of(case.k, d, case.dtype, False)
    with np.errstate(invalid="ignore"):
        stands = (m + codes * s)[ids]  # [n, hkv, block, d]
    slack = np.abs(stands) * float(torch.finfo(case.dtype).eps) / 2
    real = (np.arange(block) < np.array(held)[:, None])[:, None, :, None]
    unit = hsc[:, :, None, None]
    assert ((stands <= hb[:, :, None, 0] * unit + slack) | ~real).all()
    assert ((stands >= hb[:, :, None, 1] * unit - slack) | ~real).all()
    # the selection
    all_b, all_sc = np.zeros((nb, hkv, 2, d), np.int8), np.zeros((nb, hkv))
    all_b[ids], all_sc[ids] = hb, hsc
    want = oracle.select(case.q.double().numpy(), all_b, all_sc, case.tables.tolist(),
                         case.lens.tolist(), block, k)
    assert (sel.cpu().numpy() == want[0]).all() and (slens.cpu().numpy() == want[1]).all()
    assert (scores.cpu().double().numpy() == want[2]).all()
    # the attention: of each (sequence, KV head) over tiles of one KV head
    case.q = case.q.reshape(S * hkv, hq // hkv, d)
    case.k, case.v = (x.reshape(nb * hkv, 1, block, -1) for x in (case.k, case.v))
    case.Hkv = 1
    check(case, out.cpu().view(S * hkv, hq // hkv, d), tables=sel.cpu().view(S * hkv, k),
          lens=slens.cpu().flatten())


def test_bounds_do_not_follow_blocks_that_move():
    """A context is swapped out, its blocks' places go to others, and it comes back to other
    places; then it is copied.  Bounds are the places', as documented: stale until the whole
    length is given as new, or until they are copied along."""
    hkv, block, d, k, nb = 2, 8, 64, 6, 60
    lens, table = [27 * block - 3], torch.arange(27, dtype=torch.int32)[None]
    g = torch.Generator().manual_seed(3)
    make = lambda: (torch.randn(nb, hkv, block, d, generator=g) +  # noqa: E731
                    2 * torch.randn(nb, hkv, 1, d, generator=g)).bfloat16()
    kc, vc = make().to(DEV), make().to(DEV)
    host_k, host_v = (torch.zeros(27, hkv, block, d, dtype=torch.bfloat16).pin_memory()
                      for _ in range(2))
    q = torch.randn(1, 4 * hkv, d, generator=g).bfloat16()
    n = i32(lens)
    bounds = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device=DEV)
    scales = torch.zeros(nb, hkv, device=DEV)

    def pairs(a, b):
        return torch.tensor(list(zip(a, b)), dtype=torch.int64, device=DEV)

    def select(tab):
        sel, slens = i32(np.zeros((1, hkv, k))), i32(np.zeros((1, hkv)))
        scores = torch.zeros(1, hkv, tab.shape[1], device=DEV)
        pkv.select_blocks(sel, slens, scores, q.to(DEV), bounds, scales, tab.to(DEV), n, block)
        return sel, scores

    def places(sel, tab):  # in the context
        order = {int(b): i for i, b in enumerate(tab[0])}
        return [[order[t // hkv] for t in row] for row in sel[0].tolist()]

    pkv.block_bounds(bounds, scales, kc, table.to(DEV), n, n, lens[0])
    first, first_scores = select(table)
    old = list(range(27))
    pkv.kv_swap_blocks(host_k, host_v, kc, vc, pairs(old, old))
    saved_b, saved_sc = bounds[:27].clone(), scales[:27].clone()
    # another context of all the pool's places
    other = make().to(DEV)
    kc.copy_(other)
    every = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    whole = i32([nb * block])
    pkv.block_bounds(bounds, scales, kc, every, whole, whole, nb * block)
    stale_b, stale_sc = bounds.clone(), scales.clone()
    new = torch.randperm(nb, generator=g)[:27].tolist()
    back = torch.tensor([new], dtype=torch.int32)
    pkv.kv_swap_blocks(kc, vc, host_k, host_v, pairs(old, new))
    assert torch.equal(bounds, stale_b) and torch.equal(scales, stale_sc)
    assert not torch.equal(select(back)[1], first_scores)
    # copied along
    bounds[new], scales[new] = saved_b, saved_sc
    sel, scores = select(back)
    assert torch.equal(scores, first_scores) and places(sel, back) == places(first, table)
    # or made again
    bounds.copy_(stale_b)
    scales.copy_(stale_sc)
    pkv.block_bounds(bounds, scales, kc, back.to(DEV), n, n, lens[0])
    sel, scores = select(back)
    assert torch.equal(scores, first_scores) and places(sel, back) == places(first, table)
    assert torch.equal(bounds[new], saved_b) and torch.equal(scales[new], saved_sc)
    # copies of its blocks (a fork that writes): the last one gets a token, which bounds it
    # anew; a whole one needs the copy of its bounds
    free = [b for b in range(nb) if b not in new][:2]
    pkv.kv_copy_blocks(kc, vc, pairs([new[26], new[5]], free))
    fork = back.clone()
    fork[0, 26], fork[0, 5] = free
    one, more = i32([1]), i32([lens[0] + 1])
    pkv.block_bounds(bounds, scales, kc, fork.to(DEV), more, one, 1)
    hb, hsc = np.zeros((nb, hkv, 2, d), np.int8), np.zeros((nb, hkv))
    assert oracle.block_bounds(hb, hsc, kc.cpu().double().numpy(), fork.tolist(), [lens[0] + 1],
                               [lens[0] + 1], nb * block) == 0
    right = [i for i in range(27) if (bounds[fork[0, i]].cpu().numpy() == hb[fork[0, i]]).all()]
    assert right == [i for i in range(27) if i != 5]
    pkv.block_bounds(bounds, scales, kc, fork.to(DEV), more, more, lens[0] + 1)
    at = fork[0].tolist()
    assert (bounds[at].cpu().numpy() == hb[at]).all()
    assert (scales[at].cpu().double().numpy() == hsc[at]).all()
    assert pkv.device_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_tokens_with_the_same_slot_race_by_pairs(interleaved):
    """Of two tokens for one slot each pair of the key, and each 16 bytes of the value, is one of
    the two's; queries are rotated for both, and other slots are left alone."""
    T, hq, hkv, d, block, nb = 40, 4, 3, 64, 8, 4
    g = torch.Generator().manual_seed(2)
    q, key, value = (torch.randn(T, h, d, generator=g).half().to(DEV) for h in (hq, hkv, hkv))
    pos = torch.arange(T, device=DEV).int() * 3
    turns = pkv.rope_turns([10000.0 ** (-i / 24) for i in range(24)], DEV)
    slots = torch.tensor([5, 17] * (T // 2), device=DEV)
    kc, vc = (torch.full((nb, hkv, block, d), 9.0, dtype=torch.float16, device=DEV)
              for _ in range(2))
    q_out, want_q, want_k = torch.empty_like(q), torch.empty_like(q), torch.empty_like(key)
    pkv.rope(want_q, q, pos, turns, interleaved=interleaved)
    pkv.rope(want_k, key, pos, turns, interleaved=interleaved)
    pkv.rope_write(q_out, kc, vc, q, key, value, pos, turns, slots, interleaved=interleaved)
    assert pkv.device_status() == 0 and torch.equal(q_out, want_q)
    for slot in (5, 17):
        tokens = (slots == slot).nonzero().flatten()
        got = kc[slot // block, :, slot % block]
        if interleaved:
            pairs = lambda x: x[..., :48].unflatten(-1, (24, 2))  # noqa: E731
        else:
            pairs = lambda x: x[..., :48].unflatten(-1, (2, 24)).transpose(-1, -2)  # noqa: E731
        assert (pairs(want_k[tokens]) == pairs(got)).all(-1).any(0).all()
        for rows, cache in ((want_k, kc), (value, vc)):  # behind the pairs, and the values
            got = cache[slot // block, :, slot % block].unflatten(-1, (8, 8))
            mine = rows[tokens].unflatten(-1, (8, 8))
            first = 6 if rows is want_k else 0
            assert (mine == got).all(-1).any(0)[:, first:].all()
    left = torch.ones(nb * block, dtype=torch.bool, device=DEV)
    left[[5, 17]] = False
    for c in (kc, vc):
        assert (c.transpose(1, 2).reshape(nb * block, hkv, d)[left] == 9.0).all()
