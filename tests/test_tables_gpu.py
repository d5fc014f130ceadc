"""GPU: block tables, slot map and positions of a step, and releases, against
the oracle; every number must be equal."""
import random

import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import tables as oracle

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
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Loop:
    """A batch's tables on the GPU beside the oracle's lists."""

    def __init__(self, S, width, block, pool, rng):
        self.block, self.pool = block, pool
        self.stack = rng.sample(range(pool), pool)
        self.count, self.lens = pool, [0] * S
        self.tables = [[-1] * width for _ in range(S)]
        self.d = dict(tables=i32(self.tables), lens=i32(self.lens), stack=i32(self.stack),
                      count=i32([pool]))
        self.ws = torch.empty(pkv.tables_workspace_bytes(S), dtype=torch.uint8, device=DEV)

    def extend(self, new, rows, positions=True, in_place=True):
        d, S = self.d, len(new)
        qs = torch.full((S + 1,), 99, dtype=torch.int32, device=DEV)
        slots = torch.full((rows,), 99, dtype=torch.int64, device=DEV)
        pos = torch.full((rows,), 99, dtype=torch.int32, device=DEV) if positions else None
        lens, count = (None, None) if in_place else (d["lens"].clone(), d["count"].clone())
        pkv.tables_extend(d["tables"], d["lens"], i32(new), d["stack"], d["count"], self.block, qs,
                          slots, pos, self.ws, lens_out=lens, free_count_out=count)
        if not in_place:
            assert d["lens"].tolist() == self.lens and int(d["count"]) == self.count
            d["lens"], d["count"] = lens, count
        want = oracle.extend(self.tables, self.lens, new, self.stack, self.count, self.block,
                             self.pool, rows)
        self.lens, self.count, start, wslots, wpos, refused, bad = want
        assert qs.tolist() == start and slots.tolist() == wslots
        assert pos is None or pos.tolist() == wpos
        self.check()
        return refused, bad

    def release(self, done):
        d = self.d
        pkv.tables_release(d["tables"], d["lens"], i32(done), d["stack"], d["count"], self.block,
                           self.ws)
        self.count, refused, bad = oracle.release(self.tables, self.lens, done, self.stack,
                                                  self.count, self.block, self.pool)
        self.check()
        return refused, bad

    def check(self):
        d = self.d
        assert d["tables"].tolist() == self.tables and d["lens"].tolist() == self.lens
        assert d["stack"].tolist() == self.stack and int(d["count"]) == self.count


@pytest.mark.parametrize("S,width,block,most", [(1, 4, 16, 20), (5, 9, 1, 7), (33, 40, 8, 30),
                                                (64, 20, 32, 100), (1500, 12, 16, 40),
                                                (3, 700, 7, 4000)])
def test_a_serving_loop(S, width, block, most):
    rng = random.Random(S)
    loop = Loop(S, width, block, S * width, rng)
    for step in range(6):
        room = [width * block - n for n in loop.lens]
        new = [min(r, rng.choice([0, 1, 1, rng.randint(0, most)])) for r in room]
        assert loop.extend(new, sum(new) + rng.choice([0, 1, 300]), step % 2 == 0,
                           step % 3 != 2) == (False, False)
        assert loop.release([int(rng.random() < 0.3) for _ in range(S)]) == (False, False)
    assert pkv.device_status() == 0


def test_idle_sequences_and_no_rows():
    loop = Loop(7, 3, 8, 21, random.Random(0))
    loop.extend([0] * 7, 0)
    loop.extend([0] * 7, 5)
    loop.extend([0, 0, 24, 0, 0, 1, 0], 25)  # a full table; leading and trailing idle ones
    loop.release([0] * 7)
    assert pkv.device_status() == 0


def test_a_step_without_room_changes_nothing():
    loop = Loop(4, 6, 8, 10, random.Random(1))
    assert loop.extend([8, 9, 0, 1], 40) == (False, False)
    assert loop.extend([40, 9, 8, 0], 80)[0]       # 5 + 1 + 1 blocks of 6 free
    assert pkv.device_status() == 32
    assert loop.extend([1, 1, 1, 1], 3)[0]         # four rows of three
    assert pkv.device_status() == 32
    assert loop.extend([32, 0, 0, 0], 32) == (False, False)  # 4 of 6
    assert loop.extend([0, 0, 16, 0], 16) == (False, False)  # the last two
    assert loop.extend([0, 0, 1, 0], 1)[0]
    assert pkv.device_status() == 32


def test_bad_lengths_give_no_tokens():
    loop = Loop(4, 2, 8, 8, random.Random(2))
    for lens, new in (([3, -1, 4, 0], [2, 1, 13, 1]), ([3, 2, 17, 0], [-1, 1, 1, 16]),
                      ([0, 0, 0, 0], [2 ** 31 - 1, 1, -2 ** 31, 17])):
        loop.lens = list(lens)
        loop.tables = [[6, 7] for _ in range(4)]
        loop.d["lens"], loop.d["tables"] = i32(lens), i32(loop.tables)
        loop.stack, loop.count = [0, 1, 2, 3, 4, 5, 6, 7], 6
        loop.d["stack"], loop.d["count"] = i32(loop.stack), i32([6])
        assert loop.extend(new, 20) == (False, True)
        assert pkv.device_status() == 2


def test_bad_blocks_and_counts():
    loop = Loop(2, 3, 8, 6, random.Random(3))
    loop.stack = [0, 1, 2, 3, 9, -5]
    loop.d["stack"] = i32(loop.stack)
    loop.extend([8, 12], 20)  # the bad ids come off first
    assert pkv.device_status() == 1
    for count in (7, -1):
        loop.count = count
        loop.d["count"] = i32([count])
        assert loop.extend([1, 0], 1)[0]
        assert pkv.device_status() == 32
        if count > 0:  # nothing fits on the stack
            assert loop.release([1, 1])[0]
            assert pkv.device_status() == 32
    loop.count = 5
    loop.d["count"] = i32([5])
    assert loop.release([1, 1])[0]  # 3 blocks back onto 5 of 6
    assert pkv.device_status() == 32


def test_release_of_bad_lengths():
    loop = Loop(3, 2, 8, 6, random.Random(4))
    loop.extend([3, 9, 16], 28)
    loop.lens = [3, 17, -1]
    loop.d["lens"] = i32(loop.lens)
    assert loop.release([1, 1, 1]) == (False, True)
    assert pkv.device_status() == 2


def test_slots_match_the_host_allocators():
    S, block, pool = 9, 16, 80
    rng = random.Random(5)
    order = rng.sample(range(pool), pool)
    host = pkv.BlockAllocator(pool, block, order)
    lens = [rng.randint(1, 100) for _ in range(S)]
    for s in range(S):
        host.add(s, lens[s])
    loop = Loop(S, 8, block, pool, rng)
    loop.stack = order[::-1]
    loop.d["stack"] = i32(loop.stack)
    loop.extend(lens, sum(lens))
    host_tables, host_lens = host.dense_tables(range(S), 8)
    assert torch.equal(loop.d["tables"].cpu(), host_tables)
    assert torch.equal(loop.d["lens"].cpu(), host_lens)
    slots, pairs = host.step_append(range(S))
    before = loop.lens[:]
    loop.extend([1] * S, S)
    got = [loop.tables[s][before[s] // block] * block + before[s] % block for s in range(S)]
    assert len(pairs) == 0 and got == slots.tolist()


def test_captured_steps_share_a_workspace():
    """Two graphs (an extend and a release) on one workspace, replayed in turn:
    each replay is a step of its own."""
    S, block = 40, 8
    loop = Loop(S, 10, block, 500, random.Random(6))
    d = loop.d
    new, done = i32([1 + s % 3 for s in range(S)]), i32([0] * S)
    rows = int(new.sum()) + 4
    qs = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(rows, dtype=torch.int64, device=DEV)
    pos = torch.zeros(rows, dtype=torch.int32, device=DEV)
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        pkv.tables_extend(d["tables"], d["lens"], new, d["stack"], d["count"], block, qs, slots,
                          pos, loop.ws)
    with torch.cuda.graph(b):
        pkv.tables_release(d["tables"], d["lens"], done, d["stack"], d["count"], block, loop.ws)
    loop.check()  # capturing ran nothing
    for step in range(12):
        a.replay()
        loop.lens, loop.count, start, wslots, wpos, refused, bad = oracle.extend(
            loop.tables, loop.lens, new.tolist(), loop.stack, loop.count, block, 500, rows)
        assert not refused and not bad
        assert slots.tolist() == wslots and pos.tolist() == wpos and qs.tolist() == start
        gone = [int((s + step) % 11 == 0) for s in range(S)]
        done.copy_(i32(gone))
        b.replay()
        loop.count, _, _ = oracle.release(loop.tables, loop.lens, gone, loop.stack, loop.count,
                                          block, 500)
        loop.check()
    assert pkv.device_status() == 0
