"""GPU: the first rotation, bounds, selection and attention over selected blocks that a process
makes may be calls that a graph captures, on a stream and threads of their own."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import threading
import torch
import paged_kv_cache_312_gb300 as pkv

dev, S, Hq, Hkv, D, B, W, K = "cuda", 9, 64, 2, 128, 16, 40, 7
gen = torch.Generator(dev).manual_seed(0)
randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev).bfloat16()
i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=dev)
nb = S * W
turns = pkv.rope_turns([10000.0 ** (-i / 64) for i in range(64)], dev)
table = torch.randperm(nb, device=dev).to(torch.int32).view(S, W)
lens = torch.randint(1, W * B + 1, (S,), device=dev).to(torch.int32)
x, pos = randn(S, Hq + 2 * Hkv, D), lens - 1
slots = (table.gather(1, (pos // B).long()[:, None])[:, 0].long() * B + pos % B)
k, v = randn(nb, Hkv, B, D), randn(nb, Hkv, B, D)


def state():
    return dict(q=torch.zeros(S, Hq, D, device=dev).bfloat16(), k=k.clone(), v=v.clone(),
                b=torch.zeros(nb, Hkv, 2, D, dtype=torch.int8, device=dev),
                sc=torch.zeros(nb, Hkv, device=dev), sel=i32(S, Hkv, K), n=i32(S, Hkv),
                scores=torch.zeros(S, Hkv, W, device=dev), out=torch.zeros(S, Hq, D, device=dev),
                back=torch.zeros(S, Hq, D, device=dev).bfloat16(),
                split=torch.zeros(S, Hq, D, device=dev), ws=torch.zeros(
                    pkv.decode_workspace_bytes(S, Hq, D, K * B, 32), dtype=torch.uint8, device=dev))


def run(s, stream=None):
    q, key, value = x.split([Hq, Hkv, Hkv], 1)
    pkv.rope_write(s["q"], s["k"], s["v"], q, key, value, pos, turns, slots, stream=stream)
    pkv.rope(s["back"], s["q"], pos, turns, inverse=True, stream=stream)
    pkv.block_bounds(s["b"], s["sc"], s["k"], table, lens, lens, W * B, stream=stream)
    pkv.select_blocks(s["sel"], s["n"], s["scores"], s["q"], s["b"], s["sc"], table, lens, B,
                      stream=stream)
    pkv.paged_decode_attention_selected(s["out"], s["q"], s["k"], s["v"], s["sel"], s["n"], 0.1, B,
                                        Hkv, stream=stream)
    pkv.paged_decode_attention_selected(s["split"], s["q"], s["k"], s["v"], s["sel"], s["n"], 0.1,
                                        B, Hkv, 32, s["ws"], stream=stream)


a, c = state(), state()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run(a)
graph.replay()
run(c)
torch.cuda.synchronize()
assert all(torch.equal(a[n], c[n]) for n in a) and pkv.device_status() == 0
assert float((c["split"] - c["out"]).abs().max()) < 1e-3
assert float((c["back"].float() - x[:, :Hq].float()).abs().max()) < 0.1
# threads, each with a stream and a state of its own, at once
many, errors = [state() for _ in range(4)], []


def work(s):
    try:
        stream = torch.cuda.Stream()
        for _ in range(20):
            run(s, stream)
        stream.synchronize()
    except Exception as e:
        errors.append(e)


torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(s,)) for s in many]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
assert all(torch.equal(a[n], s[n]) for n in a for s in many) and pkv.device_status() == 0
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
