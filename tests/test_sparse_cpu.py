"""Block-sparse decode attention on the CPU: the oracle against what it promises, and the
refusals of the calls."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import sparse as oracle

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("size", [1e-30, 1e-3, 1.0, 37.5, 1e9, 1e18])
def test_oracle_bounds_hold_every_key_and_every_score(size):
    rng = np.random.default_rng(3)
    keys = rng.standard_normal((16, 64)) * size
    bounds, scale = oracle.tile_bounds(keys)
    if np.abs(keys).max() > 127 * 2.0 ** 50:
        assert scale == math.inf and not bounds.any()
        return
    wide = bounds.astype(np.float64) * scale
    assert (wide[0] >= keys.max(0)).all() and (wide[1] <= keys.min(0)).all()
    assert scale == 2.0 ** -50 or np.abs(keys).max() > 127 * scale / 2
    q = np.round(rng.standard_normal((3, 64)) * 40).clip(-127, 127)  # whole numbers: no rounding
    score = oracle.block_scores(q, bounds[None], np.array([scale]))[0]
    # no key of 16 normals lies 8 of their sizes from another, and either bound is rounded by a unit
    assert score >= (q @ keys.T).max()
    assert score <= (q @ keys.T).max() + 64 * 127 * (8 * size + 2 * scale)


@pytest.mark.parametrize("most,e", [
    (0.0, -50), (127.0, 0), (127.0000001, 1), (254.0, 1), (63.5, -1), (3.96875, -5),
    (127 * 2.0 ** 50, 50), (127 * 2.0 ** 50 * (1 + 2 ** -20), 51), (math.inf, 51), (math.nan, 51),
    (127 * 2.0 ** -50, -50), (128 * 2.0 ** -50, -49), (1e-40, -50)])
def test_oracle_exponents(most, e):
    assert oracle.exponent(most) == e


def test_oracle_selects_the_best_set():
    """Against every set of the right size: the kept blocks in it, and no other set's scores
    better, the lowest blocks of equal ones."""
    rng = np.random.default_rng(1)
    q = rng.standard_normal((1, 2, 64))
    bounds = rng.integers(-3, 4, (9, 1, 2, 64)).astype(np.int8)
    bounds[4], bounds[6] = bounds[2], bounds[2]
    scales = np.ones((9, 1))
    table = [list(rng.permutation(9))]
    for k, first, recent in itertools.product(range(1, 10), range(3), range(1, 4)):
        if first + recent > k:
            continue
        got, lens, scores, _ = oracle.select(q, bounds, scales, table, [71], 8, k, first, recent)
        order = [table[0].index(t) for t in got[0, 0] if t >= 0]
        assert order == sorted(order) and len(order) == min(k, 9)
        assert set(range(first)) | set(range(9 - recent, 9)) <= set(order)
        assert lens[0, 0] == sum(min(8, 71 - 8 * i) for i in order)
        row = oracle.block_scores(q[0], bounds[table[0], 0], scales[table[0], 0])
        free = [i for i in order if first <= i < 9 - recent]
        if k < 9:
            options = itertools.combinations(range(first, 9 - recent), len(free))
            best = max(options, key=lambda c: (sorted(row[list(c)])[::-1], [-i for i in c]))
            assert tuple(free) == best


def test_oracle_attention_over_all_blocks_is_the_dense_one():
    import oracle as dense
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(12, 2, 8, 64, generator=g) for _ in range(2))
    q = torch.randn(2, 6, 64, generator=g)
    table = torch.tensor([[3, 1, 7, 0], [5, 2, -1, -1]], dtype=torch.int32)
    lens = torch.tensor([27, 16], dtype=torch.int32)
    want = dense.paged_decode_attention(q, k, v, table, lens, 0.125, 8, 2)
    bounds, scales = np.zeros((12, 2, 2, 64), np.int8), np.zeros((12, 2))
    sel, slens, _, _ = oracle.select(q.numpy(), bounds, scales, table.tolist(), lens, 8, 4)
    got = oracle.attention(q.numpy(), k.numpy(), v.numpy(), sel, slens, 0.125)
    assert np.abs(got - want).max() < 1e-12


# ---- refusals --------------------------------------------------------------------------------

def bounds(b=256, sc=256, kc=256, bt=256, lens=256, new=256, S=4, W=8, NB=64, Hkv=2, D=128, B=16,
           most=1, dtype=2):
    return pkv.lib().pkv_block_bounds(P(b), P(sc), P(kc), P(bt), P(lens), P(new), S, W, NB, Hkv, D,
                                      B, most, dtype, P(0))


def select(sel=256, slens=256, scores=256, q=256, b=256, sc=256, bt=256, lens=256, S=4, Hq=8,
           Hkv=2, D=128, B=16, W=8, NB=64, K=4, first=1, recent=1, dtype=2):
    return pkv.lib().pkv_select_blocks(P(sel), P(slens), P(scores), P(q), P(b), P(sc), P(bt),
                                       P(lens), S, Hq, Hkv, D, B, W, NB, K, first, recent, dtype,
                                       P(0))


def attend(q4=False, out=256, q=256, kc=256, vc=256, sel=256, slens=256, scale=0.1, B=16, Hkv=2,
           S=4, Hq=8, D=128, K=4, NB=64, dtype=2, out_dtype=2, part=0, ws=0, wb=0):
    name = "pkv_paged_decode_attention_selected" + ("_q4" if q4 else "")
    return getattr(pkv.lib(), name)(P(out), P(q), P(kc), P(vc), P(sel), P(slens), scale, B, Hkv, S,
                                    Hq, D, K, NB, dtype, out_dtype, part, P(ws), wb, P(0))


@pytest.mark.parametrize("call", [bounds, select])
@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -3), (dict(S=-1), -2), (dict(S=65536), -2), (dict(S=0), 0), (dict(W=0), -2),
    (dict(NB=0), -2), (dict(Hkv=0), -2), (dict(Hkv=65536), -2), (dict(D=96), -2),
    (dict(B=12), -2), (dict(W=1 << 27), -2), (dict(NB=1 << 27), -2), (dict(b=0), -1),
    (dict(sc=0), -1), (dict(bt=0), -1), (dict(lens=0), -1), (dict(b=264), -10),
    (dict(sc=258), -10), (dict(bt=258), -10), (dict(lens=258), -10), (dict(S=0, bt=0), 0)])
def test_refusals(call, change, code):
    assert call(**change) == code
    if code:
        assert call.__name__.encode() in pkv.lib().pkv_last_error_string()


@pytest.mark.parametrize("change,code", [
    (dict(most=-1), -2), (dict(most=(1 << 30) + 1), -2), (dict(most=0), 0), (dict(new=0), -1),
    (dict(new=258), -10), (dict(kc=0), -1), (dict(kc=264), -10),
    (dict(S=65535, W=1 << 20, B=8, Hkv=128, most=1 << 23), -2)])
def test_bounds_refusals(change, code):
    assert bounds(**change) == code


@pytest.mark.parametrize("change,code", [
    (dict(Hq=0), -2), (dict(Hq=7), -2), (dict(Hq=65536), -2), (dict(Hq=258), -4),
    (dict(first=-1), -2), (dict(recent=0), -2), (dict(first=3, recent=2), -2), (dict(K=1), -2),
    (dict(K=(1 << 30) + 1), -2), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), -2),
    (dict(sel=0), -1), (dict(slens=0), -1), (dict(scores=0), -1), (dict(q=0), -1),
    (dict(q=264), -10), (dict(sel=258), -10), (dict(slens=258), -10), (dict(scores=258), -10)])
def test_select_refusals(change, code):
    assert select(**change) == code


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), -3), (dict(out_dtype=5), -3), (dict(S=-1), -2), (dict(S=0), 0),
    (dict(S=32768), -2), (dict(S=32767, NB=1 << 26), -2), (dict(Hq=7), -2), (dict(D=96), -2),
    (dict(B=12), -2), (dict(K=0), -2), (dict(NB=0), -2), (dict(K=1 << 27), -2),
    (dict(scale=math.inf), -2), (dict(part=8), -2), (dict(part=32), -8), (dict(out=0), -1),
    (dict(q=0), -1), (dict(kc=0), -1), (dict(vc=0), -1), (dict(sel=0), -1), (dict(slens=0), -1),
    (dict(kc=264), -10), (dict(vc=264), -10), (dict(ws=264, wb=1 << 20), -10),
    (dict(ws=256, wb=16), -8)])
def test_attention_refusals(q4, change, code):
    assert attend(q4, **change) == code
    if code:
        assert b"attention_selected" in pkv.lib().pkv_last_error_string()


def test_attention_over_4_bits_takes_16_bit_queries():
    assert attend(True, dtype=0) == -4


def test_binding_refusals():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    f = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    b, sc = torch.zeros(9, 2, 2, 64, dtype=torch.int8), torch.zeros(9, 2)
    calls = {
        pkv.block_bounds: ([b, sc, f(9, 2, 16, 64), i(3, 4), i(3), i(3), 1], [
            (0, b.to(torch.uint8)), (0, b[:, :1]), (1, sc.double()), (1, sc[:8]),
            (2, f(9, 2, 16, 32)), (3, i(2, 4)), (4, i(3).long()), (5, i(2))]),
        pkv.select_blocks: ([i(3, 2, 4), i(3, 2), torch.zeros(3, 2, 8), f(3, 4, 64), b, sc,
                             i(3, 8), i(3), 16], [
            (0, i(3, 1, 4)), (0, i(3, 4)), (1, i(3)), (2, torch.zeros(3, 2, 7)),
            (2, torch.zeros(3, 2, 8).half()), (3, f(3, 4, 32)), (3, f(2, 4, 64)), (4, b[:8]),
            (6, i(2, 8)), (7, i(3).long())]),
        pkv.paged_decode_attention_selected: (
            [f(3, 4, 64), f(3, 4, 64), f(9, 2, 16, 64), f(9, 2, 16, 64), i(3, 2, 4), i(3, 2), 0.1,
             16, 2], [
                (0, f(3, 4, 32)), (1, f(3, 4, 64).half()), (2, f(9, 2, 16, 32)), (3, f(8, 2, 16, 64)),
                (4, i(3, 4)), (4, i(3, 2, 4).long()), (5, i(3)), (7, 8), (8, 4)])}
    for call, (good, changes) in calls.items():
        for at, bad in [(None, None)] + changes:
            a = list(good)
            if at is not None:
                a[at] = bad
            with pytest.raises(ValueError):  # the good ones are host tensors
                call(*a)


# ---- calls as words --------------------------------------------------------------------------

LAYOUTS = {1: ("pkv_rope", "_ROPE"), 2: ("pkv_rope_write", "_ROPE_WRITE"),
           3: ("pkv_block_bounds", "_BLOCK_BOUNDS"), 4: ("pkv_select_blocks", "_SELECT_BLOCKS"),
           5: ("pkv_paged_decode_attention_selected", "_ATTENTION_SELECTED"),
           6: ("pkv_paged_decode_attention_selected_q4", "_ATTENTION_SELECTED")}


@pytest.mark.parametrize("call", sorted(LAYOUTS))
def test_words_reach_the_call_as_arguments_do(call):
    """Each argument in turn set to a value that the call refuses or takes: the same code and
    message either way (the message names the value)."""
    from paged_kv_cache_312_gb300 import _binding
    name, layout = LAYOUTS[call]
    layout, types = getattr(_binding, layout), _binding._SIGS[name][1]
    fn = getattr(pkv.lib(), name)
    at_axis = 4 if name == "pkv_rope" else 8 if name == "pkv_rope_write" else None
    good = {1: [256] * 4 + [None, 1, 0, 8, 128, 128, 1024, 1024, 1.0, 0, 0, 2, 0],
            2: [256] * 8 + [None, 1, 256, 0, 1024, 1024, 256, 256, 9, 8, 2, 128, 128, 16, 1.0, 0, 2, 0],
            3: [256] * 6 + [0, 8, 64, 2, 128, 16, 1, 2, 0],
            4: [256] * 8 + [0, 8, 2, 128, 16, 8, 64, 4, 1, 1, 2, 0],
            5: [256] * 6 + [0.1, 16, 2, 0, 8, 128, 4, 64, 2, 2, 0, 0, 0, 0],
            6: [256] * 6 + [0.1, 16, 2, 0, 8, 128, 4, 64, 2, 2, 0, 0, 0, 0]}[call]
    assert len(good) == len(types)
    for at in [None] + list(range(len(good))):
        args = list(good)
        if at is not None:
            args[at] = b"\7" * 64 if at == at_axis else math.nan if args[at].__class__ is float else -77
        if types[at or 0] is ctypes.c_void_p and at not in (None, at_axis):
            args[at] = 0
        want = (fn(*args), pkv.lib().pkv_last_error_string())
        words = layout.pack(call, *[x for i, x in enumerate(args) if i != at_axis])
        got = (pkv.lib().pkv_call_words(words, None if at_axis is None else args[at_axis]),
               pkv.lib().pkv_last_error_string())
        assert got == want, (name, at)


def test_words_refusals():
    call = pkv.lib().pkv_call_words
    words = lambda *x: b"".join(int(i).to_bytes(8, "little", signed=True) for i in x)  # noqa: E731
    assert call(None, None) == -1
    assert call(words(0), None) == -2 and call(words(7), None) == -2
    assert call(words(3, *[256] * 6, 2 ** 32, 8, 64, 2, 128, 16, 1, 2, 0), None) == -2
    assert b"32 bits" in pkv.lib().pkv_last_error_string()
    assert call(words(3, *[256] * 6, 0, 8, 64, 2, 128, 16, 1, 2, 0), None) == 0
