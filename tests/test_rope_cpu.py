"""Rotary positions on the CPU: the oracle against the definition, the turns, the refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import rope as oracle

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("base,pairs", [(10000.0, 32), (500000.0, 64), (1e6, 8)])
def test_turns_are_the_rounded_fractions(base, pairs):
    freq = [base ** (-i / pairs) for i in range(pairs)] + [0.0, 1e-12, 3.5, -1.0, 2.0 ** 20,
                                                           2 * math.pi, 1e-300]
    got = pkv.rope_turns(freq).tolist()
    # two doubles of 1 / (2 pi) and one rounding at the end: within a unit of 2^-64 (of a frequency
    # past 1, of 2^-106 of the turns too)
    for g, w, f in zip(got, oracle.turns(freq), freq):
        off = (g - w + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= 1, (f, off)


def test_turns_refusals():
    lib = pkv.lib()
    one, out = (ctypes.c_double * 1)(1.0), (ctypes.c_int64 * 1)(7)
    assert lib.pkv_rope_turns(one, -1, out) == -2
    assert lib.pkv_rope_turns(None, 1, out) == -1 and lib.pkv_rope_turns(one, 1, None) == -1
    assert lib.pkv_rope_turns(None, 0, None) == 0
    for bad in (float("nan"), float("inf"), 2.0 ** 21, -2.0 ** 21):
        assert lib.pkv_rope_turns((ctypes.c_double * 1)(bad), 1, out) == -2 and out[0] == 7
    with pytest.raises(ValueError):
        pkv.rope_turns([[1.0]])
    with pytest.raises(pkv.PkvError):
        pkv.rope_turns([math.nan])


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_is_a_rotation_of_complex_numbers(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 48))
    freq = np.array([10.0 ** (-i / 4) for i in range(16)])
    pos = np.array([[0, 1, 17, 1000, 5], [3, 3, 2, 1, 0]])
    axis = [i % 2 for i in range(16)]
    angle = oracle.angles(pos, oracle.turns(freq), axis)
    y = oracle.rope(x, angle, interleaved, magnitude=0.5)
    a, b = oracle.pairs_of(32, interleaved)
    want = (x[..., a] + 1j * x[..., b]) * 0.5 * np.exp(1j * (pos[axis].T * freq))[:, None]
    # angles up to 1000 radians in doubles: 1000 * 2^-53 each way
    assert np.allclose(y[..., a] + 1j * y[..., b], want, atol=1e-11)
    assert (y[..., 32:] == x[..., 32:]).all()
    back = oracle.rope(y, angle, interleaved, inverse=True, magnitude=2.0)
    assert np.allclose(back, x, atol=1e-14)


# ---- refusals --------------------------------------------------------------------------------

def rope(out=256, x=256, pos=256, turns=256, axis=None, axes=1, T=4, H=8, D=128, R=128, os=1024,
         xs=1024, m=1.0, dtype=2):
    return pkv.lib().pkv_rope(P(out), P(x), P(pos), P(turns), axis, axes, T, H, D, R, os, xs, m, 0,
                              0, dtype, P(0))


def write(q_out=256, kc=256, vc=256, q=256, key=256, value=256, pos=256, turns=256, axis=None,
          axes=1, slots=256, T=4, qos=1024, qs=1024, ks=256, vs=256, NB=9, Hq=8, Hkv=2, D=128,
          R=128, B=16, m=1.0, dtype=2):
    return pkv.lib().pkv_rope_write(P(q_out), P(kc), P(vc), P(q), P(key), P(value), P(pos),
                                    P(turns), axis, axes, P(slots), T, qos, qs, ks, vs, NB, Hq,
                                    Hkv, D, R, B, m, 0, dtype, P(0))


BOTH = [
    (dict(dtype=3), -3), (dict(D=0), -2), (dict(D=72), -2), (dict(D=272, R=16), -2),
    (dict(R=0), -2), (dict(R=24), -2), (dict(R=144), -2), (dict(axes=0), -2), (dict(axes=5), -2),
    (dict(axes=2), -1), (dict(axes=2, axis=bytes([2] * 64)), -2), (dict(axis=bytes([1] * 64)), -2),
    (dict(T=-1), -2), (dict(T=0), 0), (dict(pos=0), -1), (dict(turns=0), -1), (dict(pos=258), -10),
    (dict(turns=260), -10), (dict(m=math.nan), -2), (dict(m=math.inf), -2)]


@pytest.mark.parametrize("call", [rope, write])
@pytest.mark.parametrize("change,code", BOTH)
def test_refusals(call, change, code):
    assert call(**change) == code
    if code:
        assert b"pkv_rope" in pkv.lib().pkv_last_error_string()


@pytest.mark.parametrize("change,code", [
    (dict(H=0), -2), (dict(H=65536), -2), (dict(x=0), -1), (dict(out=0), -1), (dict(x=264), -10),
    (dict(out=264), -10), (dict(xs=1016), -2), (dict(xs=1028), -2), (dict(os=1016), -2),
    (dict(os=2048), -2), (dict(x=0, T=0), 0)])
def test_rope_refusals(change, code):
    assert rope(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(Hq=-1), -2), (dict(Hkv=0), -2), (dict(Hkv=65536), -2), (dict(NB=-1), -2),
    (dict(B=0), -2), (dict(NB=1 << 26), -2), (dict(q=0), -1), (dict(q_out=0), -1),
    (dict(key=0), -1), (dict(value=0), -1), (dict(kc=0), -1), (dict(vc=0), -1), (dict(slots=0), -1),
    (dict(q=264), -10), (dict(q_out=264), -10), (dict(key=264), -10), (dict(value=264), -10),
    (dict(kc=264), -10), (dict(vc=264), -10), (dict(slots=260), -10), (dict(qs=1016), -2),
    (dict(qos=1020), -2), (dict(ks=248), -2), (dict(vs=260), -2), (dict(qos=2048), -2),
    (dict(T=0, kc=0), 0)])
def test_rope_write_refusals(change, code):
    assert write(**change) == code


def test_binding_refusals():
    f = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    pos, turns = torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)
    good = [f(3, 4, 64), f(3, 4, 64), pos, turns]
    for at, bad in ((None, None), (0, f(3, 4, 32)), (0, f(3, 4, 64).float()), (2, pos.long()),
                    (2, pos[:2]), (2, pos[0]), (2, pos[None, None]), (3, turns.int()),
                    (3, turns[None]), (0, f(3, 4)), (1, f(3, 4))):
        a = list(good)
        if at is not None:
            a[at] = bad
        with pytest.raises(ValueError):  # the good ones are host tensors
            pkv.rope(*a)
    cache, slots = f(2, 4, 16, 64), torch.zeros(3, dtype=torch.int64)
    good = [f(3, 8, 64), cache, cache, f(3, 8, 64), f(3, 4, 64), f(3, 4, 64), pos, turns, slots]
    for at, bad in ((None, None), (0, None), (1, f(2, 4, 16, 32)), (3, f(3, 8, 32)),
                    (3, f(24, 64)), (4, f(3, 2, 64)), (4, f(12, 64)), (4, f(3, 4, 64).half()),
                    (8, slots.int()), (8, slots[:2])):
        a = list(good)
        if at is not None:
            a[at] = bad
        with pytest.raises(ValueError):
            pkv.rope_write(*a)
