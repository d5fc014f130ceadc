"""GPU: rows rotated, and rotated on the way into the cache, against the oracle.

A row's element is off by at most (|a| + |b|) m 2^-21 before it is rounded: the angle's float
(2^-25 of pi), two units in the last place of sincospi (2^-23), the magnitude (2^-24) and a
product and a fused sum (2^-24 each) are 2^-25 pi + 2^-23 + 3 * 2^-24 < 2^-21."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import rope as oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def rows(t, h, d, dtype, seed):
    return torch.randn(t, h, d, generator=torch.Generator().manual_seed(seed)).to(dtype)


def freqs(rotary, base=10000.0):
    return [base ** (-2 * i / rotary) for i in range(rotary // 2)]


def places(t, axes, far, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (axes, t), generator=g, dtype=torch.int32)


def check(got, x, angle, interleaved, inverse=False, magnitude=1.0):
    """got (device) against the oracle's rotation of x (host)."""
    want = oracle.rope(x.double().numpy(), angle, interleaved, inverse, magnitude)
    rotary, fin = 2 * angle.shape[1], torch.finfo(x.dtype)
    size = np.zeros_like(want)
    a, b = oracle.pairs_of(rotary, interleaved)
    both = (np.abs(x.double().numpy()[..., a]) + np.abs(x.double().numpy()[..., b])) * abs(magnitude)
    size[..., a] = size[..., b] = both * 2.0 ** -21
    size += np.maximum(np.abs(want) + size, float(fin.smallest_normal)) * fin.eps / 2
    size[..., rotary:] = 0
    off = np.abs(got.cpu().double().numpy() - want)
    assert (off <= size).all(), float((off / np.maximum(size, 1e-300)).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,h,d,rotary,axes,interleaved", [
    (1, 1, 16, 16, 1, False), (1, 3, 64, 64, 1, True), (4, 8, 64, 32, 1, False),
    (33, 5, 80, 80, 1, True), (7, 64, 128, 128, 3, False), (19, 2, 96, 48, 2, True),
    (5, 9, 256, 256, 4, False), (3, 71, 128, 16, 1, True), (300, 1, 128, 112, 1, False)])
def test_rope_matches_the_oracle(dtype, t, h, d, rotary, axes, interleaved):
    x, pos = rows(t, h, d, dtype, t), places(t, axes, 1 << 20, d)
    units = pkv.rope_turns(freqs(rotary))
    pairs = rotary // 2
    axis = [i * axes // pairs for i in range(pairs)] if axes > 1 else None
    angle = oracle.angles(pos.numpy(), units.tolist(), axis)
    dx, dpos, dt = x.to(DEV), (pos if axes > 1 else pos[0]).to(DEV), units.to(DEV)
    for inverse, magnitude in ((False, 1.0), (True, 1.25)):
        out = torch.full_like(dx, 77.0)
        pkv.rope(out, dx, dpos, dt, axis, interleaved, inverse, magnitude)
        check(out, x, angle, interleaved, inverse, magnitude)
    again = dx.clone()
    pkv.rope(again, again, dpos, dt, axis, interleaved, True, 1.25)
    assert torch.equal(again, out) and torch.equal(dx.cpu(), x)
    assert pkv.device_status() == 0


def test_positions_of_any_size_turn_exactly():
    pos = torch.tensor([[0, 1, -1, -12345, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]],
                       dtype=torch.int32)
    freq = freqs(64) [:28] + [0.0, 2 * math.pi, 100.0, -0.5]
    units = pkv.rope_turns(freq)
    x = rows(8, 2, 64, torch.float32, 1)
    out = torch.empty_like(x, device=DEV)
    pkv.rope(out, x.to(DEV), pos.to(DEV), units.to(DEV))
    check(out, x, oracle.angles(pos.numpy(), units.tolist()), False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,hq,hkv,d,rotary,block,axes,interleaved,fused", [
    (1, 1, 1, 64, 64, 8, 1, False, False), (1, 32, 32, 128, 128, 16, 1, False, True),
    (64, 8, 1, 128, 64, 16, 1, True, True), (150, 6, 2, 80, 80, 5, 3, False, True),
    (77, 0, 3, 64, 32, 32, 1, True, False), (41, 16, 8, 256, 192, 16, 2, False, False)])
def test_rope_write_matches_the_oracle(dtype, t, hq, hkv, d, rotary, block, axes, interleaved,
                                       fused):
    nb = -(-t // block) + 3
    g = torch.Generator().manual_seed(t)
    x = rows(t, hq + 2 * hkv, d, dtype, 5)
    q, key, value = x.split([hq, hkv, hkv], 1)
    slots = torch.randperm(nb * block, generator=g)[:t].to(torch.int64)
    slots[3::5] = -1
    pos, pairs = places(t, axes, 131072, 9), rotary // 2
    axis = [(axes - 1) - i * axes // pairs for i in range(pairs)] if axes > 1 else None
    units = pkv.rope_turns(freqs(rotary, 500000.0))
    angle = oracle.angles(pos.numpy(), units.tolist(), axis)
    kc, vc = (torch.full((nb, hkv, block, d), 3.0, dtype=dtype, device=DEV) for _ in range(2))
    dx = x.to(DEV)
    dq, dk, dv = dx.split([hq, hkv, hkv], 1)
    if not fused:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    q_out = torch.full((t, hq, d), 5.0, dtype=dtype, device=DEV)
    pkv.rope_write(q_out if hq else None, kc, vc, dq if hq else None, dk, dv, pos.to(DEV),
                   units.to(DEV), slots.to(DEV), axis, interleaved, 0.75)
    assert pkv.device_status() == 0
    live = slots >= 0
    if hq:
        check(q_out[live.to(DEV)], q[live], angle[live.numpy()], interleaved, False, 0.75)
        assert (q_out[~live.to(DEV)] == 5).all()
    at, offset = slots[live] // block, slots[live] % block
    check(kc.cpu()[at, :, offset].to(DEV), key[live], angle[live.numpy()], interleaved, False, 0.75)
    assert torch.equal(vc.cpu()[at, :, offset], value[live])
    rest = torch.ones(nb, block, dtype=torch.bool)
    rest[at, offset] = False
    for c in (kc, vc):
        assert (c.cpu().transpose(1, 2)[rest] == 3).all()
    assert torch.equal(dx.cpu(), x)
    if hq:  # in place, among the other rows of the projection
        pkv.rope_write(dq, kc, vc, dq, dk, dv, pos.to(DEV), units.to(DEV), slots.to(DEV), axis,
                       interleaved, 0.75)
        assert torch.equal(dq[live.to(DEV)], q_out[live.to(DEV)])
        assert torch.equal(dq.cpu()[~live], q[~live])
        if fused:
            assert torch.equal(dx.cpu()[:, hq:], x[:, hq:])


def test_bad_slots_are_flagged_and_left_out():
    nb, hkv, block, d = 3, 2, 8, 64
    kc = torch.zeros(nb, hkv, block, d, device=DEV)
    vc = torch.zeros_like(kc)
    x = torch.ones(3, hkv, d, device=DEV)
    q_out = torch.full((3, hkv, d), 9.0, device=DEV)
    slots = torch.tensor([nb * block, 5, 1 << 40], device=DEV)
    pkv.rope_write(q_out, kc, vc, x, x, x, torch.zeros(3, dtype=torch.int32, device=DEV),
                   pkv.rope_turns(freqs(64), DEV), slots)
    assert pkv.device_status() == 4
    assert (q_out[[0, 2]] == 9).all() and (q_out[1] == 1).all()
    assert (vc[0, :, 5] == 1).all() and float(vc.sum()) == hkv * d


def test_no_tokens():
    x = torch.zeros(0, 2, 64, device=DEV)
    pos, units = torch.zeros(0, dtype=torch.int32, device=DEV), pkv.rope_turns(freqs(64), DEV)
    pkv.rope(x, x.clone(), pos, units)
    kc = torch.zeros(1, 2, 8, 64, device=DEV)
    pkv.rope_write(None, kc, kc.clone(), None, x, x, pos, units,
                   torch.zeros(0, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(interleaved):
    """Of the formula by autograd in 64 bits, and of the kernel by differences: the rotation is
    linear, so a difference of any width is the derivative."""
    t, h, d, rotary = 6, 3, 64, 48
    x, w = rows(t, h, d, torch.float32, 1), rows(t, h, d, torch.float32, 2)
    pos, units = places(t, 1, 4096, 3), pkv.rope_turns(freqs(rotary))
    angle = torch.from_numpy(oracle.angles(pos.numpy(), units.tolist()))[:, None]
    leaf = x.double().requires_grad_()
    a, b = (torch.from_numpy(i) for i in oracle.pairs_of(rotary, interleaved))
    first = leaf[..., a] * angle.cos() - leaf[..., b] * angle.sin()
    second = leaf[..., b] * angle.cos() + leaf[..., a] * angle.sin()
    (1.5 * ((first * w[..., a]).sum() + (second * w[..., b]).sum()) +
     (leaf[..., rotary:] * w[..., rotary:]).sum()).backward()
    grad = torch.empty_like(x, device=DEV)
    args = (pos.to(DEV), units.to(DEV), None, interleaved)
    pkv.rope(grad, w.to(DEV), *args, inverse=True, magnitude=1.5)
    # (|a| + |b|) m 2^-21 and the fp32 rounding, of normals below 6
    assert float((grad.cpu().double() - leaf.grad).abs().max()) <= 12 * 1.5 * 2.0 ** -20

    def loss(v):
        y = torch.empty_like(v)
        pkv.rope(y, v, *args, magnitude=1.5)
        return float((y.double() * w.to(DEV).double()).sum())

    base, step = x.to(DEV), 4.0
    for i in range(0, t * h * d, 131):
        up, down = base.clone(), base.clone()
        up.view(-1)[i] += step
        down.view(-1)[i] -= step
        # two elements of each row's pair are off by 2^-20 of it, times w
        assert abs((loss(up) - loss(down)) / (2 * step) - float(grad.view(-1)[i])) < 1e-3


def test_another_stream_and_a_captured_call():
    t, hq, hkv, d, block, nb = 37, 8, 4, 128, 16, 5
    x = rows(t, hq + 2 * hkv, d, torch.bfloat16, 3).to(DEV)
    q, key, value = x.split([hq, hkv, hkv], 1)
    pos, units = places(t, 1, 999, 3)[0].to(DEV), pkv.rope_turns(freqs(d), DEV)
    slots = torch.randperm(nb * block, device=DEV)[:t]
    kc = torch.zeros(nb, hkv, block, d, dtype=torch.bfloat16, device=DEV)
    sets = [[torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV), kc.clone(), kc.clone()]
            for _ in range(3)]
    call = lambda s, **k: pkv.rope_write(*s, q, key, value, pos, units, slots, **k)  # noqa: E731
    call(sets[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(sets[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(sets[2])
    pos.add_(1)
    graph.replay()
    pos.sub_(1)
    graph.replay()
    torch.cuda.synchronize()
    for s in sets[1:]:
        assert all(torch.equal(a, b) for a, b in zip(sets[0], s))
    with pytest.raises(ValueError):
        pkv.rope(q[..., ::2], q[..., ::2], pos, units)
    with pytest.raises(pkv.PkvError):  # one row for all tokens: refused, not read as 37
        pkv.rope(torch.zeros_like(sets[0][0]), q[:1].expand(t, hq, d), pos, units)


def test_rows_past_2_31_elements():
    """A strided tensor whose last rows start beyond 2^31 elements: 4.3 GB."""
    h, d, stride = 1, 64, 1 << 16
    t = (1 << 31) // stride + 3
    base = torch.zeros(t * stride, dtype=torch.bfloat16, device=DEV)
    x = base.view(t, stride)[:, :h * d].unflatten(1, (h, d))
    x.copy_(torch.randn(t, h, d, device=DEV))
    pos, units = places(t, 1, 999, 3), pkv.rope_turns(freqs(d))
    last = x[-8:].cpu()
    pkv.rope(x, x, pos[0].to(DEV), units.to(DEV))
    check(x[-8:], last, oracle.angles(pos[:, -8:].numpy(), units.tolist()), False)
