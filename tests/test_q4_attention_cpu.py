"""Refusals of the 4-bit decode attention (nothing is launched), and the oracle
against a direct softmax."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_312_gb300 as pkv
from oracle import q4

P = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def attend(out=256, q=256, k=256, bt=256, scale=0.1, B=16, Hkv=2, S=3, Hq=8, D=128, W=8, NB=64, kv=2,
           od=0, part=0, ws=0, wb=0):
    return pkv.lib().pkv_paged_decode_attention_q4(
        P(out), P(q), P(k), P(256), P(bt), P(256), scale, B, Hkv, S, Hq, D, W, NB, kv, od, part,
        P(ws), wb, P(0))


@pytest.mark.parametrize("change,code", [
    (dict(kv=0), -4), (dict(kv=5), -3), (dict(od=9), -3), (dict(S=-1), -2), (dict(S=70000), -2),
    (dict(D=96), -2), (dict(B=4), -2), (dict(Hq=7), -2), (dict(Hkv=0), -2), (dict(W=0), -2),
    (dict(NB=0), -2), (dict(part=24), -2), (dict(part=-16), -2), (dict(scale=float("nan")), -2),
    (dict(NB=1 << 27), -2), (dict(W=1 << 27), -2), (dict(out=0), -1), (dict(q=0), -1),
    (dict(k=0), -1), (dict(bt=0), -1), (dict(k=264), -10), (dict(q=258), -10), (dict(out=258), -10),
    (dict(part=16), -8), (dict(part=16, ws=256, wb=100), -8), (dict(ws=256, wb=100), -8),
    (dict(ws=264, wb=1 << 20), -10), (dict(part=16, ws=264, wb=1 << 20), -10),
    (dict(S=0, out=0, k=0), 0), (dict(bt=258), -10)])
def test_refusals(change, code):
    assert attend(**change) == code
    if code:
        assert b"pkv_paged_decode_attention_q4" in pkv.lib().pkv_last_error_string()


def test_binding_refusals():
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 16, 72, dtype=torch.uint8)
    bt, cl = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = [q.clone(), q, k, k, bt, cl, 0.1, 16, 2]
    for at, bad in ((None, None), (0, q[:2]), (1, q[..., :64]), (2, k.float()), (3, k[:2]),
                    (4, bt[:2]), (4, bt.long()), (5, cl[:2]), (7, 8), (8, 4), (1, q.double())):
        a = list(good)
        if at is not None:
            a[at] = bad
        with pytest.raises(ValueError):  # the good ones are host tensors
            pkv.paged_decode_attention_q4(*a)


def test_oracle_is_attention_over_the_values():
    g = torch.Generator().manual_seed(1)
    x, y = (torch.randn(20, 2, 64, generator=g).half() for _ in range(2))
    k = torch.zeros(5, 2, 8, 36, dtype=torch.uint8)
    v = k.clone()
    table = torch.tensor([[3, 0, 4], [1, -1, 2]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, p // 8]) * 8 + p % 8 for p in range(20)])
    q4.kv_write(k, v, x, y, slots)
    q = torch.randn(2, 4, 64, generator=g).half()
    out = q4.paged_decode_attention(q, k, v, table, [20, 0], 0.2)
    K, V = q4.kv_read(k, v, slots, 64, torch.float16)
    for h in range(4):
        p = np.exp(K[:, h // 2] @ q[0, h].double().numpy() * 0.2)
        assert np.allclose(out[0, h], p @ V[:, h // 2] / p.sum(), rtol=1e-12, atol=1e-14)
    assert not out[1].any()
    hidden = q4.paged_decode_attention(q, k, v, table, [8, 24], 0.2)  # the middle block is hidden
    K, V = q4.values(k, 64, torch.float16, False), q4.values(v, 64, torch.float16, True)
    K, V = (np.concatenate([t[1, 0], t[2, 0]]) for t in (K, V))
    p = np.exp(K @ q[1, 1].double().numpy() * 0.2)
    assert np.allclose(hidden[1, 1], p @ V / p.sum(), rtol=1e-12, atol=1e-14)
