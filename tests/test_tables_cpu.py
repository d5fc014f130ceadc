"""Block tables on the GPU, on the CPU: the oracle against the host allocator
(which hands out and takes back blocks in the same order), and the refusals."""
import ctypes
import random

import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import tables as oracle

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("seed", range(6))
def test_oracle_hands_out_the_host_allocators_blocks(seed):
    rng = random.Random(seed)
    block, pool, S, width = rng.choice([1, 3, 8, 16]), 120, 6, 20
    order = rng.sample(range(pool), pool)
    host = pkv.BlockAllocator(pool, block, order)
    # the host's free list hands out order[0] first: the stack holds it on top
    stack, count = order[::-1], pool
    tables, lens, live = [[-1] * width for _ in range(S)], [0] * S, [False] * S
    for _ in range(40):
        new = [rng.choice([0, 1, 1, rng.randint(0, 2 * block)]) for _ in range(S)]
        new = [min(n, width * block - old) for n, old in zip(new, lens)]
        lens, count, start, slots, pos, refused, bad = oracle.extend(
            tables, lens, new, stack, count, block, pool, sum(new) + 3)
        assert not refused and not bad
        want = []
        for s in range(S):
            if not live[s]:
                host.add(s, 0)
                live[s] = True
            for _ in range(new[s]):
                want.append(host.append(s)[0])
        assert slots == want + [-1] * 3
        assert start == [sum(new[:i]) for i in range(S + 1)]
        done = [int(rng.random() < 0.2) for _ in range(S)]
        count, refused, bad = oracle.release(tables, lens, done, stack, count, block, pool)
        assert not refused and not bad and count == pool - sum(-(-n // block) for n in lens)
        for s in reversed(range(S)):
            if done[s]:
                host.free(s)
                live[s] = False
        for s in range(S):
            if live[s]:
                held = -(-lens[s] // block)
                assert tables[s][:held] == host.table(s) and tables[s][held:] == [-1] * (width - held)
            else:
                assert lens[s] == 0 and tables[s] == [-1] * width


def test_oracle_release_of_what_an_extend_took_restores_the_stack():
    stack = [4, 2, 7, 0, 1, 5, 3, 6]
    tables, before = [[-1] * 4 for _ in range(3)], list(stack)
    lens, count, *_ = oracle.extend(tables, [0, 0, 0], [5, 0, 9], stack, 8, 4, 8, 14)
    assert tables[0][:2] == [6, 3] and tables[2][:3] == [5, 1, 0] and count == 3
    count, _, _ = oracle.release(tables, lens, [1, 1, 1], stack, count, 4, 8)
    assert count == 8 and stack == before and lens == [0, 0, 0]


# ---- refusals --------------------------------------------------------------------------------

def extend(S=4, W=8, B=16, NB=64, T=10, ws=256, wb=256, bt=256, slots=256, qs=256, lens=256):
    p = P(256)
    return pkv.lib().pkv_tables_extend(P(bt), P(lens), p, p, p, P(qs), P(slots), P(0), p, p, S, W, B,
                                       NB, T, P(ws), wb, P(0))


def release(S=4, W=8, B=16, NB=64, ws=256, wb=256, bt=256, lens=256):
    p = P(256)
    return pkv.lib().pkv_tables_release(P(bt), P(lens), p, p, p, S, W, B, NB, P(ws), wb, P(0))


@pytest.mark.parametrize("call", [extend, release])
@pytest.mark.parametrize("change,code", [
    (dict(S=-1), -2), (dict(S=65536, wb=1 << 20), -2), (dict(W=0), -2), (dict(B=0), -2),
    (dict(NB=0), -2), (dict(W=1 << 27, B=16), -2), (dict(bt=0), -1), (dict(lens=0), -1),
    (dict(ws=0), -8), (dict(S=64, wb=256), -8), (dict(ws=264), -10), (dict(bt=258), -10),
    (dict(lens=258), -10)])
def test_refusals(call, change, code):
    assert call(**change) == code
    assert ("pkv_tables_" + call.__name__).encode() in pkv.lib().pkv_last_error_string()


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), -2), (dict(S=0), -2), (dict(S=0, T=0, bt=0), 0), (dict(slots=0), -1),
    (dict(slots=260), -10), (dict(qs=0), -1), (dict(T=(1 << 30) + 1), -2), (dict(qs=258), -10)])
def test_extend_refusals(change, code):
    assert extend(**change) == code


def test_workspace_bytes():
    f = pkv.lib().pkv_tables_workspace_bytes
    assert f(0) == 0 and f(-3) == 0 and f(1) == 256 and f(63) == 256 and f(64) == 512
    assert f(65535) == 65536 * 4
    assert pkv.tables_workspace_bytes(1000) == 4096


def test_binding_refusals():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    good = [i(3, 4), i(3), i(3), i(9), i(1), 16, i(4), torch.zeros(5, dtype=torch.int64), i(5),
            torch.zeros(256, dtype=torch.uint8)]
    for at, bad in ((None, None), (0, i(2, 4)), (1, i(3).long()), (2, i(4)), (4, i(2)), (6, i(3)),
                    (7, i(5)), (8, i(4))):
        a = list(good)
        if at is not None:
            a[at] = bad
        with pytest.raises(ValueError):  # the good ones are host tensors
            pkv.tables_extend(*a)
    rel = [good[0], good[1], i(3), good[3], good[4], 16, good[9]]
    for at, bad in ((None, None), (0, i(3)), (2, i(4)), (2, i(3).bool()), (4, i(2))):
        a = list(rel)
        if at is not None:
            a[at] = bad
        with pytest.raises(ValueError):
            pkv.tables_release(*a)
