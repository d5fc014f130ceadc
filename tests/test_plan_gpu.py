"""GPU: every row of a planned 16-bit decode call is written, whatever the lengths.

Outputs start as NaN; inputs are unit normals, so that the error allowed is the
16-bit calls' own, 2e-3 against the oracle (weights rounded once to the cache's
type: half a step, 2^-9 of bf16, of a mean of values near 1 over hundreds of
tokens)."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_312_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    pkv.device_status(reset=True)


def batch(lens, Hq, Hkv, D, B, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // B) for n in lens]
    nb = sum(need) + 2
    order = torch.randperm(nb, generator=g).int()
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(nb, Hkv, B, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(len(lens), Hq, D, generator=g).to(dtype)
    return q, k, v, tables, torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("lens,P", [
    ([8192, 2000, 5000, 3100], 512),        # a partition a warp, four to a CTA
    ([8192, 300, 0, 7000, 1, 4096] * 6, 512),
    ([4096, 100, 2000, 900] * 9, 256),      # more sequences than a warp has lanes
    ([8192, 2000, 5000, 3100], 1024),       # a partition a CTA
    ([8000, 8192, 7900, 8100], 512),        # near-equal: pieces
    ([8192, 2000, 5000, 3100] * 10, 0)])    # not split: the order alone
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (32, 4)])
def test_every_row_of_a_planned_call_is_written(lens, P, Hq, Hkv):
    B, D = 16, 64
    q, k, v, tables, cl = batch(lens, Hq, Hkv, D, B, torch.bfloat16, len(lens) + P)
    want = oracle.paged_decode_attention(q, k, v, tables, cl, 0.125, B, Hkv,
                                         nthreads=oracle.default_threads())
    args = [t.to(DEV) for t in (q, k, v, tables, cl)]
    ws = torch.full((pkv.decode_workspace_bytes(len(lens), Hq, D, tables.shape[1] * B, P),), 0xFF,
                    dtype=torch.uint8, device=DEV)
    for _ in range(3):
        out = torch.full(q.shape, float("nan"), device=DEV)
        pkv.paged_decode_attention(out, *args, 0.125, B, Hkv, partition_size=P, workspace=ws)
        got = out.cpu().double().numpy()
        assert np.isfinite(got).all()
        assert np.abs(got - want).max() <= 2e-3
    assert pkv.device_status() == 0


@pytest.mark.parametrize("P", [2 ** 31 - 32, 1 << 30, 512])
@pytest.mark.parametrize("four_bits", [False, True])
def test_a_partition_beyond_every_context(P, four_bits):
    """One partition a context: the bits of the call that is not split."""
    Hq, Hkv, D, B = 16, 8, 64, 16
    q, k, v, tables, cl = batch([500, 1, 0, 333], Hq, Hkv, D, B, torch.float16, 3)
    call = pkv.paged_decode_attention
    if four_bits:
        rows = [x.transpose(1, 2).reshape(-1, Hkv, D).to(DEV) for x in (k, v)]
        k = torch.zeros(pkv.q4_cache_shape(k.shape[0], Hkv, B, D), dtype=torch.uint8, device=DEV)
        v = torch.zeros_like(k)
        pkv.kv_write_q4(k, v, *rows, torch.arange(k.shape[0] * B, device=DEV))
        call = pkv.paged_decode_attention_q4
    args = [t.to(DEV) for t in (q, k, v, tables, cl)]
    outs = []
    for split in (0, P):
        ws = torch.empty(pkv.decode_workspace_bytes(4, Hq, D, tables.shape[1] * B, split),
                         dtype=torch.uint8, device=DEV)
        outs.append(torch.full(q.shape, float("nan"), device=DEV))
        call(outs[-1], *args, 0.125, B, Hkv, partition_size=split, workspace=ws)
    assert torch.equal(*outs) and pkv.device_status() == 0
