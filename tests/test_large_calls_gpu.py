"""GPU: the forms that only large calls of the 4-bit cache and of the block tables
take, against the oracles: writes of two stretches a warp, steps and releases in two
launches that are refused or find bad lengths, more requests than a CTA keeps in
shared memory, and a 4-bit history brought back for the 16-bit prefill."""
import random

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_312_gb300 as pkv
from oracle import q4
from test_q4_attention_gpu import Case, check
from test_tables_gpu import Loop, i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


@pytest.mark.parametrize("dtype,block,d", [(torch.bfloat16, 16, 128), (torch.float16, 32, 128),
                                           (torch.float16, 8, 64), (torch.bfloat16, 32, 64)])
@pytest.mark.parametrize("scattered", [False, True])
def test_large_writes_match_the_oracle_byte_for_byte(dtype, block, d, scattered):
    """160,008 rows of K: above the 77,824 (head_dim 128) or 155,648 (64) from which a
    warp takes two stretches; an odd number of tokens, some of them padding."""
    t, hkv = 20001, 8
    nb = -(-t // block) + 40
    g = torch.Generator().manual_seed(d + block)
    key, value = (torch.randn(t, hkv, d, generator=g) *
                  (torch.randn(t, hkv, 1, generator=g) * 2).exp() for _ in range(2))
    key, value = key.to(dtype), value.to(dtype)
    slots = torch.randperm(nb * block, generator=g)[:t] if scattered else torch.arange(t) + 7
    slots[3::11] = -1
    k = torch.randint(0, 256, pkv.q4_cache_shape(nb, hkv, block, d), generator=g, dtype=torch.uint8)
    v = torch.randint(0, 256, k.shape, generator=g, dtype=torch.uint8)
    dk, dv, ds = k.to(DEV), v.to(DEV), slots.to(DEV)
    pkv.kv_write_q4(dk, dv, key.to(DEV), value.to(DEV), ds)
    q4.kv_write(k, v, key, value, slots)
    for got, want in ((dk.cpu(), k), (dv.cpu(), v)):
        assert torch.equal(got, want), "%d bytes differ" % int((got != want).sum())
    back = [torch.full((t, hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    pkv.kv_read_q4(*back, dk, dv, ds)
    fin, hidden = torch.finfo(dtype), (slots < 0).numpy()
    for got, want in zip(back, q4.kv_read(k, v, slots, d, dtype)):
        got = got.cpu().double().numpy()
        assert (got[hidden] == 7).all()
        got, want = got[~hidden], want[~hidden]
        # half a step of the fused multiply-add in fp32 and of the type
        size = np.maximum(np.abs(want), float(fin.smallest_normal))
        assert (np.abs(got - want) <= size * (fin.eps / 2 + 2.0 ** -24) * (1 + 1e-9)).all()
    assert pkv.device_status() == 0


@pytest.mark.parametrize("S,most", [(5000, 1), (5000, 40), (4095, 9), (4096, 9), (2049, 1)])
def test_steps_of_thousands_of_requests(S, most):
    rng = random.Random(S + most)
    loop = Loop(S, 4, 16, 3 * S, rng)
    for step in range(3):
        room = [4 * 16 - n for n in loop.lens]
        new = [min(r, rng.randint(0, most)) for r in room]
        assert loop.extend(new, sum(new) + 5, step % 2 == 0, step % 2 == 0) == (False, False)
        assert loop.release([int(rng.random() < 0.3) for _ in range(S)]) == (False, False)
    assert pkv.device_status() == 0


@pytest.mark.parametrize("S", [70, 1500, 5000])
def test_a_large_step_without_room_changes_nothing(S):
    """More than 2048 rows: the scan and the rows are kernels of their own."""
    loop = Loop(S, 8, 8, 5 * S, random.Random(S))
    rows = 64 * S
    assert loop.extend([32] * S, rows, in_place=False) == (False, False)   # 4 of 5 blocks each
    assert loop.extend([17] * S, rows)[0]                                  # 3 more, and 1 is there
    assert pkv.device_status() == 32
    assert loop.extend([17] * S, rows, positions=False, in_place=False)[0]
    assert pkv.device_status() == 32
    assert loop.extend([2] * S, max(2 * S - 1, 2049))[0] == (2 * S - 1 >= 2049)  # a row too few
    assert pkv.device_status() == (32 if 2 * S - 1 >= 2049 else 0)
    assert loop.extend([1] * S, rows) == (False, False)
    loop.count = 5 * S + 1
    loop.d["count"] = i32([loop.count])
    assert loop.extend([1] * S, rows)[0]
    assert pkv.device_status() == 32


@pytest.mark.parametrize("S", [200, 5000])
def test_a_large_release_without_room_changes_nothing(S):
    """More than 1024 table entries: the scan and the rows are kernels of their own."""
    loop = Loop(S, 8, 8, 5 * S, random.Random(S))
    loop.extend([32] * S, 32 * S)
    loop.count += 1  # one place of the stack too few
    loop.d["count"] = i32([loop.count])
    assert loop.release([1] * S)[0]
    assert pkv.device_status() == 32
    loop.count = -1
    loop.d["count"] = i32([-1])
    assert loop.release([1] * S)[0]
    assert pkv.device_status() == 32
    loop.count = S
    loop.d["count"] = i32([S])
    assert loop.release([1] * S) == (False, False)
    assert pkv.device_status() == 0


@pytest.mark.parametrize("S", [300, 5000])
def test_bad_lengths_in_large_calls(S):
    loop = Loop(S, 8, 8, 8 * S, random.Random(S))
    loop.extend([20] * S, 20 * S)
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        loop.lens[S // 3] = bad
        loop.d["lens"] = i32(loop.lens)
        assert loop.extend([9] * S, 9 * S, in_place=bad < 0) == (False, True)
        assert pkv.device_status() == 2
        loop.lens[S // 3] = 20
        done = [int(s % 2 == 0 or s == S // 3) for s in range(S)]
        loop.lens[S // 3] = bad
        loop.d["lens"] = i32(loop.lens)
        assert loop.release(done) == (False, True)
        assert pkv.device_status() == 2


@pytest.mark.parametrize("S", [4, 300])
def test_bad_table_entries_are_given_back_as_they_are(S):
    """Flagged when they are given back, and again when a step takes them."""
    loop = Loop(S, 4, 8, 4 * S, random.Random(S))
    loop.extend([20] * S, 20 * S)
    assert pkv.device_status() == 0
    for s, id in ((0, -7), (S // 2, 4 * S), (S - 1, 2 ** 31 - 1)):
        loop.tables[s][s % 3] = id
    loop.d["tables"] = i32(loop.tables)
    assert loop.release([1] * S) == (False, False)
    assert pkv.device_status() == 1
    assert loop.extend([20] * S, 20 * S) == (False, False)
    assert pkv.device_status() == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_4_bit_history_under_a_16_bit_prefill(dtype):
    """A prompt chunk attends over a history held in 4 bits: its rows are read back,
    written into the blocks of a 16-bit pool, and the chunk's own after them."""
    Hq, Hkv, d, block = 8, 2, 128, 16
    past, chunk = [100, 0, 37, 16], [20, 5, 1, 40]
    S = len(past)
    g = torch.Generator().manual_seed(1)
    need = [-(-(a + b) // block) for a, b in zip(past, chunk)]
    nb, width = sum(need) + 2, max(need)
    order = torch.randperm(nb, generator=g).int()
    tables = torch.full((S, width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    slot = lambda s, p: int(tables[s, p // block]) * block + p % block  # noqa: E731
    old = torch.tensor([slot(s, p) for s in range(S) for p in range(past[s])])
    new = torch.tensor([slot(s, p) for s in range(S) for p in range(past[s], past[s] + chunk[s])])
    rows = [torch.randn(len(old), Hkv, d, generator=g).to(dtype).to(DEV) for _ in range(2)]
    k4 = torch.zeros(pkv.q4_cache_shape(nb, Hkv, block, d), dtype=torch.uint8, device=DEV)
    v4 = torch.zeros_like(k4)
    pkv.kv_write_q4(k4, v4, *rows, old.to(DEV))

    k, v = (torch.full((nb, Hkv, block, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    back = [torch.empty_like(r) for r in rows]
    pkv.kv_read_q4(*back, k4, v4, old.to(DEV))
    pkv.kv_write(k, v, *back, old.to(DEV))
    fresh = [torch.randn(len(new), Hkv, d, generator=g).to(dtype).to(DEV) for _ in range(2)]
    pkv.kv_write(k, v, *fresh, new.to(DEV))
    q = torch.randn(len(new), Hq, d, generator=g).to(dtype)
    lens = torch.tensor([a + b for a, b in zip(past, chunk)], dtype=torch.int32)
    start = torch.tensor([0] + list(np.cumsum(chunk)), dtype=torch.int32)
    out = torch.full(q.shape, float("nan"), device=DEV)
    pkv.paged_prefill_attention(out, q.to(DEV), k, v, tables.to(DEV), lens.to(DEV), start.to(DEV),
                                d ** -0.5, block, Hkv, max_query_len=max(chunk))

    hk, hv = (torch.zeros(nb, Hkv, block, d, dtype=dtype) for _ in range(2))
    want_rows = [torch.from_numpy(r).to(dtype) for r in q4.kv_read(k4.cpu(), v4.cpu(), old, d, dtype)]
    oracle.kv_write(hk, hv, *want_rows, old, block)
    oracle.kv_write(hk, hv, *(f.cpu() for f in fresh), new, block)
    want = oracle.paged_prefill_attention(q, hk, hv, tables, lens, start, d ** -0.5, block, Hkv,
                                          nthreads=oracle.default_threads())
    # unit normals: the prefill's weights are rounded once to 16 bits
    assert np.abs(out.cpu().double().numpy() - want).max() <= 2e-3
    assert pkv.device_status() == 0


@pytest.mark.parametrize("rise", [0.0, 30.0])
@pytest.mark.parametrize("power", [78, -100])
def test_values_of_any_size_that_is_allowed(power, rise):
    """Values near 2^80, and far below the normal numbers of fp16, under scores that
    stay and that climb."""
    def key(k):
        return k + torch.linspace(0, rise, k.shape[0])[:, None, None]

    case = Case(torch.bfloat16, 8, 2, 128, 16, [700, 3], k=key, q=lambda q: q.abs() * 0.3,
                v=lambda v: v.clamp(-4, 4) * 2.0 ** power)
    for P in (0, 64):
        check(case, case.run(P=P))
