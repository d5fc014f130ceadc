"""GPU: the first call that a process makes may be one that a graph captures: nothing
of the library has run or been loaded before."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import torch
import paged_kv_cache_312_gb300 as pkv

dev, S, Hq, Hkv, D, B, width, nb = "cuda", 100, 64, 8, 128, 16, 20, 2000
i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=dev)
tables, lens, count = i32(S, width).fill_(-1), i32(S), i32(1).fill_(nb)
stack, new, qs = torch.arange(nb, dtype=torch.int32, device=dev), i32(S).fill_(30), i32(S + 1)
done = i32(S)
slots = torch.zeros(30 * S, dtype=torch.int64, device=dev)
gen = torch.Generator(dev).manual_seed(0)
randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev).bfloat16()
key, value, q = randn(30 * S, Hkv, D), randn(30 * S, Hkv, D), randn(S, Hq, D)
k4 = torch.zeros(S * width, Hkv, B, 9 * D // 16, dtype=torch.uint8, device=dev)
v4 = torch.zeros_like(k4)
k, v = (torch.zeros(nb, Hkv, B, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
back = [torch.zeros_like(key) for _ in range(2)]
tws = torch.zeros(4096, dtype=torch.uint8, device=dev)
outs = [torch.zeros(S, Hq, D, device=dev) for _ in range(6)]
ws = torch.zeros(1 << 26, dtype=torch.uint8, device=dev)


def run():
    pkv.tables_extend(tables, lens, new, stack, count, B, qs, slots, None, tws)
    pkv.kv_write_q4(k4, v4, key, value, slots)
    pkv.kv_read_q4(back[0], back[1], k4, v4, slots)
    pkv.kv_write(k, v, key, value, slots)
    for i, (P, w) in enumerate(((0, None), (0, ws), (64, ws))):
        pkv.paged_decode_attention_q4(outs[i], q, k4, v4, tables, lens, 0.1, B, Hkv,
                                      partition_size=P, workspace=w)
        pkv.paged_decode_attention(outs[3 + i], q, k, v, tables, lens, 0.1, B, Hkv,
                                   partition_size=P, workspace=w)
    pkv.tables_release(tables, lens, done, stack, count, B, tws)


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
assert lens.tolist() == [30] * S and int(count) == nb - 2 * S
got = [t.clone() for t in outs + back + [k4, v4, tables]]
lens.zero_(), count.fill_(nb), tables.fill_(-1)
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs + back + [k4, v4, tables]))
assert float((outs[0] - outs[2]).abs().max()) < 2e-2 and float(outs[0].abs().max()) > 0.1
assert pkv.device_status() == 0
print("captured first")
"""


def test_a_process_may_capture_its_first_calls():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
