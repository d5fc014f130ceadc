"""GPU: writing into the 4-bit cache, reading it back and moving its blocks,
against the oracle.  Bytes must match bit for bit; rows read back match what
the bytes stand for, rounded once to the cache's type."""
import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import q4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def pools(nb, hkv, block, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(0, 256, pkv.q4_cache_shape(nb, hkv, block, d), generator=g, dtype=torch.uint8)
    return k, torch.randint(0, 256, k.shape, generator=g, dtype=torch.uint8)


def rows(t, hkv, d, dtype, seed=1):
    """Normals with runs of very different sizes and offsets."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, hkv, d // 64, 64, generator=g)
    x = x * (torch.randn(t, hkv, d // 64, 1, generator=g) * 3).exp()
    x = x + torch.randn(t, hkv, d // 64, 1, generator=g)
    return x.reshape(t, hkv, d).to(dtype)


def same_bytes(got, want):
    got = got.cpu()
    assert torch.equal(got, want), "%d bytes differ" % int((got != want).sum())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("block,d,hkv,t", [(8, 64, 1, 1), (8, 64, 3, 77), (16, 128, 8, 150),
                                           (32, 128, 2, 64), (16, 64, 5, 33), (32, 64, 2, 2),
                                           (8, 128, 1, 3)])
def test_write_matches_the_oracle_byte_for_byte(dtype, block, d, hkv, t):
    nb = 23
    k, v = pools(nb, hkv, block, d)
    key, value = rows(t, hkv, d, dtype, 1), rows(t, hkv, d, dtype, 2)
    g = torch.Generator().manual_seed(t)
    for scattered in (True, False):
        slots = torch.randperm(nb * block, generator=g)[:t] if scattered else torch.arange(t) + 5
        slots = slots.to(torch.int64)
        slots[::7] = -1 if t > 1 else slots[0]
        dk, dv = k.to(DEV), v.to(DEV)
        pkv.kv_write_q4(dk, dv, key.to(DEV), value.to(DEV), slots.to(DEV))
        wk, wv = k.clone(), v.clone()
        q4.kv_write(wk, wv, key, value, slots)
        same_bytes(dk, wk)
        same_bytes(dv, wv)
    assert pkv.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_write_of_ties_and_extreme_runs(dtype):
    """Runs on a grid of whole codes and halves (every tie), of equal elements,
    with the type's greatest and least values, with spreads that round to a
    scale of zero or below the normal numbers, and with NaN and infinities."""
    d, hkv = 64, 1
    fin = torch.finfo(dtype)
    grid = torch.arange(64, dtype=torch.float64)
    runs = [grid / 4 % 16, (grid % 31) / 2, -(grid % 31) / 2, grid * 0 + 3.25, grid * 0,
            torch.where(grid < 32, fin.max / 4, -fin.max / 4), torch.where(grid < 5, fin.max, 0.0),
            grid * fin.smallest_normal / 64, grid * fin.smallest_normal, grid * fin.smallest_normal * 7,
            torch.where(grid == 0, -1000.0, grid / 1024), 100 + (grid % 2) / 2]
    for scale in (3.0, 1 / 7, 1e-3):
        runs += [(grid % 31) / 2 * scale, (grid % 31 - 15) / 2 * scale + 1]
    x = torch.stack(runs).to(dtype).reshape(-1, hkv, d)
    odd = x[:3].clone()
    odd[0, 0, 5], odd[1, 0, 63], odd[2, 0, 0] = float("nan"), float("inf"), -float("inf")
    t = x.shape[0]
    k, v = pools(4, hkv, 8, d)
    slots = torch.randperm(32, generator=torch.Generator().manual_seed(4))[:t].to(torch.int64)
    dk, dv = k.to(DEV), v.to(DEV)
    pkv.kv_write_q4(dk, dv, x.to(DEV), x.flip(0).to(DEV), slots.to(DEV))
    q4.kv_write(k, v, x, x.flip(0), slots)
    same_bytes(dk, k)
    same_bytes(dv, v)
    pkv.kv_write_q4(dk, dv, odd.to(DEV), odd.to(DEV), slots[:3].to(DEV))
    got = q4.kv_read(dk.cpu(), dv.cpu(), slots[:3], d, dtype)
    assert all(np.isnan(g).all() for g in got)
    back = torch.zeros(3, hkv, d, dtype=dtype, device=DEV)
    pkv.kv_read_q4(back, back.clone(), dk, dv, slots[:3].to(DEV))
    assert torch.isnan(back).all()
    assert pkv.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_write_of_elements_far_below_the_minimum(dtype):
    """x - m is a tie but for an x (or m) that fp32 loses beside the other, or
    nearly does: the code is that of the exact difference."""
    tiny = [2.0 ** -e for e in range(12, 25)]
    runs = []
    for size in (1.0, 0.125, 8.0):
        for sign in (-1.0, 1.0):
            for start in (0, 7):  # all of them, and beside the grid's ties
                x = (torch.arange(64, dtype=torch.float64) % 16 - 7.5) * size
                x[20:20 + len(tiny)] = torch.tensor(tiny, dtype=torch.float64) * sign
                x[50:50 + start] = 0.0
                runs.append(x)
    for e in (14, 20, 24):  # an m of almost nothing beside whole codes and halves
        for sign in (-1.0, 1.0):
            x = torch.arange(64, dtype=torch.float64) % 31 / 2 + 1
            x[3] = 2.0 ** -e * sign
            x[5] = 15.0
            runs.append(x)
    x = torch.stack(runs).to(dtype).reshape(len(runs), 1, 64)
    k, v = pools(3, 1, 8, 64)
    slots = torch.arange(len(runs))
    dk, dv = k.to(DEV), v.to(DEV)
    pkv.kv_write_q4(dk, dv, x.to(DEV), x.flip(0).to(DEV), slots.to(DEV))
    q4.kv_write(k, v, x, x.flip(0), slots)
    same_bytes(dk, k)
    same_bytes(dv, v)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("block,d,hkv,t", [(8, 64, 3, 50), (16, 128, 4, 1), (32, 128, 2, 131)])
def test_read_matches_the_oracle(dtype, block, d, hkv, t):
    nb = 9
    g = torch.Generator().manual_seed(3)
    k, v = pools(nb, hkv, block, d)
    allslots = torch.arange(nb * block)
    q4.kv_write(k, v, rows(nb * block, hkv, d, dtype, 4), rows(nb * block, hkv, d, dtype, 5), allslots)
    slots = torch.randint(0, nb * block, (t,), generator=g)  # repeats among them
    slots[3::5] = -1
    key = torch.full((t, hkv, d), 7.0, dtype=dtype, device=DEV)
    value = key.clone()
    pkv.kv_read_q4(key, value, k.to(DEV), v.to(DEV), slots.to(DEV))
    for got, want in zip((key, value), q4.kv_read(k, v, slots, d, dtype)):
        want = np.where((slots < 0).numpy()[:, None, None], 7.0, want)
        got = got.cpu().double().numpy()
        # m + c s in fp32 (one rounding of a fused multiply-add), then the type: half a step of
        # each, relative to the value but at least to the least normal number
        fin = torch.finfo(dtype)
        size = np.maximum(np.abs(want), float(fin.smallest_normal))
        assert (np.abs(got - want) <= size * (fin.eps / 2 + 2.0 ** -24) * (1 + 1e-9)).all()
    assert pkv.device_status() == 0


def test_rows_of_a_fused_projection_and_other_streams():
    t, hkv, d, block, nb = 37, 4, 128, 16, 5
    qkv = torch.randn(t, 6 + 2, hkv, d, device=DEV).to(torch.bfloat16)
    key, value = qkv[:, 6], qkv[:, 7]
    slots = torch.randperm(nb * block, device=DEV)[:t]
    a, b = (torch.zeros(pkv.q4_cache_shape(nb, hkv, block, d), dtype=torch.uint8, device=DEV)
            for _ in range(2))
    a2, b2 = a.clone(), b.clone()
    pkv.kv_write_q4(a, b, key.contiguous(), value.contiguous(), slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.kv_write_q4(a2, b2, key, value, slots, stream=side)
    side.synchronize()
    assert torch.equal(a, a2) and torch.equal(b, b2)
    with pytest.raises(ValueError):
        pkv.kv_write_q4(a, b, key[..., ::2], value[..., ::2], slots)
    with pytest.raises(pkv.PkvError):  # one row for all tokens: refused, not read as 37
        pkv.kv_write_q4(a, b, key[:1].expand(t, hkv, d), value, slots)


def test_bad_slots_are_flagged_and_skipped():
    nb, hkv, block, d = 4, 2, 16, 64
    k, v = pools(nb, hkv, block, d)
    x = torch.ones(3, hkv, d, dtype=torch.float16)
    slots = torch.tensor([nb * block, 5, 1 << 40])
    dk, dv = k.to(DEV), v.to(DEV)
    pkv.kv_write_q4(dk, dv, x.to(DEV), x.to(DEV), slots.to(DEV))
    assert pkv.device_status() == 4
    q4.kv_write(k, v, x, x, slots)
    same_bytes(dk, k)
    same_bytes(dv, v)
    out = torch.full((3, hkv, d), 9.0, dtype=torch.float16, device=DEV)
    out2 = out.clone()
    pkv.kv_read_q4(out, out2, dk, dv, slots.to(DEV))
    assert pkv.device_status() == 4
    assert (out[[0, 2]] == 9).all() and (out[1] == 1).all() and (out2[1] == 1).all()


def test_no_tokens():
    k = torch.zeros(pkv.q4_cache_shape(2, 2, 8, 64), dtype=torch.uint8, device=DEV)
    x = torch.zeros(0, 2, 64, dtype=torch.float16, device=DEV)
    s = torch.zeros(0, dtype=torch.int64, device=DEV)
    pkv.kv_write_q4(k, k.clone(), x, x, s)
    pkv.kv_read_q4(x, x.clone(), k, k.clone(), s)


def test_blocks_of_a_4_bit_pool_are_copied_and_swapped():
    k, v = pools(12, 3, 8, 64)
    dk, dv = k.to(DEV), v.to(DEV)
    pairs = torch.tensor([[0, 5], [3, 11], [1, 2]])
    pkv.kv_copy_blocks(dk, dv, pairs.to(DEV))
    for s, d in pairs.tolist():
        k[d], v[d] = k[s], v[s]
    same_bytes(dk, k)
    same_bytes(dv, v)
    hk, hv = (torch.zeros(pkv.q4_cache_shape(6, 3, 8, 64), dtype=torch.uint8).pin_memory()
              for _ in range(2))
    out = torch.tensor([[5, 0], [2, 4]], device=DEV)
    pkv.kv_swap_blocks(hk, hv, dk, dv, out)
    torch.cuda.synchronize()
    assert torch.equal(hk[[0, 4]], k[[5, 2]]) and torch.equal(hv[[0, 4]], v[[5, 2]])
    assert not hk[[1, 2, 3, 5]].any()
    assert pkv.device_status() == 0


def test_a_pool_past_2_31_bytes():
    """Blocks whose tiles start beyond 2^31 bytes: 4.8 GB a pool."""
    nb, hkv, block, d = 1 << 16, 32, 32, 128
    k = torch.empty(pkv.q4_cache_shape(nb, hkv, block, d), dtype=torch.uint8, device=DEV)
    v = torch.empty_like(k)
    x = torch.randn(4, hkv, d, device=DEV).to(torch.bfloat16)
    slots = torch.tensor([0, nb * block - 1, (nb // 2) * block + 7, nb * block - 2], device=DEV)
    pkv.kv_write_q4(k, v, x, x, slots)
    a, b = torch.empty_like(x), torch.empty_like(x)
    pkv.kv_read_q4(a, b, k, v, slots)
    last = q4.values(k[-1:].cpu(), d, torch.bfloat16, False)[0, :, [block - 1, block - 2]]
    assert torch.equal(a[[1, 3]].cpu(), torch.from_numpy(last).to(torch.bfloat16))
    assert torch.equal(a, b) and pkv.device_status() == 0
