"""The 4-bit cache on the CPU: the oracle against the format's own identities,
and the refusals of the C ABI and of the binding, which launch nothing."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import q4

P = ctypes.c_void_p
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rows(dtype, seed=0, shape=(5, 3, 128)):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.rand(shape[:-1] + (1,), generator=g).exp()
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_an_element_comes_back_within_half_a_scale(dtype):
    x = rows(dtype)
    codes, pairs = q4.quantise(x)
    s, m = (pairs[..., i].double().numpy().repeat(64, -1).reshape(5, 3, 128) for i in (0, 1))
    wide = x.double().numpy()
    # half a scale, and at code 15 what the scale's own rounding leaves: half a step of 15 s
    bound = s * (0.5 + 15 * HALF_STEP[dtype]) * (1 + 1e-9)
    assert (np.abs(m + codes * s - wide) <= bound).all()
    # the least element of each run is exact
    runs = (m + codes * s).reshape(5, 3, 2, 64)
    assert (runs.min(-1) == wide.reshape(5, 3, 2, 64).min(-1)).all()


@pytest.mark.parametrize("is_v", [False, True])
@pytest.mark.parametrize("block,d", [(8, 64), (16, 128), (32, 64)])
def test_a_tile_places_every_element_once(block, d, is_v):
    seen = set()
    for i in range(block):
        for e in range(d):
            byte, shift = q4.code_place(i, e, block, d, is_v)
            assert 0 <= byte < block * d // 2 and (byte, shift) not in seen
            seen.add((byte, shift))
    assert len(seen) == block * d
    ends = [q4.pair_place(i, block, d) for i in range(block)]
    assert ends[0].start == block * d // 2
    assert all(a.stop == b.start for a, b in zip(ends, ends[1:]))
    assert ends[-1].stop == pkv.lib().pkv_q4_tile_bytes(block, d) == block * d * 9 // 16


def test_write_then_read_gives_the_quantised_rows():
    x, y = rows(torch.bfloat16, 1), rows(torch.bfloat16, 2)
    k = torch.full((4, 3, 8, 72), 0xAB, dtype=torch.uint8)
    v = k.clone()
    slots = torch.tensor([3, 17, -1, 32, 2])
    q4.kv_write(k, v, x, y, slots)
    for got, want in zip(q4.kv_read(k, v, slots, 128, torch.bfloat16), (x, y)):
        codes, pairs = q4.quantise(want)
        p = pairs.double().numpy().repeat(64, -2).reshape(5, 3, 128, 2)
        full = p[..., 1] + codes * p[..., 0]
        keep = [0, 1, 4]  # slot -1 and slot 32 (past the pool) hold nothing
        assert (got[keep] == full[keep]).all()
    # no other byte changed
    fresh = torch.full_like(k, 0xAB)
    q4.kv_write(fresh, fresh.clone(), x[[0, 1, 4]], y[[0, 1, 4]], slots[[0, 1, 4]])
    assert torch.equal(fresh, k)


def test_runs_of_equal_or_non_finite_elements():
    x = torch.zeros(3, 1, 128, dtype=torch.float16)
    x[0] = 1.5
    x[1, 0, 3] = float("inf")
    x[2, 0, 70] = float("nan")
    codes, pairs = q4.quantise(x)
    assert (codes == 0).all()
    assert pairs[0].tolist() == [[[0.0, 1.5], [0.0, 1.5]]]
    assert torch.isnan(pairs[1, 0, 0]).all() and pairs[1, 0, 1].tolist() == [0.0, 0.0]
    assert torch.isnan(pairs[2, 0, 1]).all() and pairs[2, 0, 0].tolist() == [0.0, 0.0]


# ---- refusals --------------------------------------------------------------------------------

def write(T=3, ks=256, vs=256, NB=4, H=2, D=128, B=16, dt=2, k=256, key=256, slots=8):
    return pkv.lib().pkv_kv_write_q4(P(k), P(256), P(key), P(256), P(slots), T, ks, vs, NB, H, D,
                                     B, dt, P(0))


def read(T=3, NB=4, H=2, D=128, B=16, dt=2, k=256, key=256, slots=8):
    return pkv.lib().pkv_kv_read_q4(P(key), P(256), P(k), P(256), P(slots), T, NB, H, D, B, dt,
                                    P(0))


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("change,code", [
    (dict(dt=7), -3), (dict(dt=0), -4), (dict(D=96), -2), (dict(B=12), -2), (dict(T=-1), -2),
    (dict(NB=-1), -2), (dict(H=0), -2), (dict(k=0), -1), (dict(key=0), -1), (dict(slots=0), -1),
    (dict(k=264), -10), (dict(key=264), -10), (dict(slots=12), -10), (dict(T=0, k=0), 0),
    (dict(NB=1 << 26), -2), (dict(H=65536), -2), (dict(T=1 << 30, H=8), -2)])
def test_cache_refusals(call, change, code):
    assert call(**change) == code
    if code:
        assert call.__name__.encode() in pkv.lib().pkv_last_error_string()


@pytest.mark.parametrize("change", [dict(ks=255), dict(vs=248), dict(ks=260), dict(ks=0)])
def test_write_refuses_strides(change):
    assert write(**change) == -2


def test_tile_bytes_of_sizes_outside_the_format():
    f = pkv.lib().pkv_q4_tile_bytes
    assert f(8, 64) == 288 and f(32, 128) == 2304 and f(4, 64) == 0 and f(16, 96) == 0
    assert pkv.q4_cache_shape(7, 2, 16, 128) == (7, 2, 16, 72)
    with pytest.raises(ValueError):
        pkv.q4_cache_shape(7, 2, 12, 128)


def test_binding_refusals():
    k = torch.zeros(4, 2, 16, 72, dtype=torch.uint8)
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for a in ([k, k, x, x, slots],                          # host tensors
              [k.float(), k, x, x, slots], [k, k[:3], x, x, slots],
              [k, k, x[:, :1], x[:, :1], slots], [k, k, x, x.half(), slots],
              [k, k, x, x, slots.int()], [k, k, x, x, slots[:2]],
              [k, k, x[..., :64], x[..., :64], slots]):
        with pytest.raises(ValueError):
            pkv.kv_write_q4(*a)
        with pytest.raises(ValueError):
            pkv.kv_read_q4(a[2], a[3], a[0], a[1], a[4])
