"""CPU: what the selection of blocks and the split attention over selected tiles launch.
native/select_launches.cpp compiles them as they are over stand-ins for the CUDA runtime."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from paged_kv_cache_312_gb300 import build as product

NATIVE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "select_launches.cpp")
SOURCES = ("block_select.cu", "selected_split.cu")
DEFAULT_LIMIT = 48 * 1024  # static and dynamic shared memory of a kernel that sets none
MOST = 227 * 1024          # of a CTA


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    out = tmp_path_factory.mktemp("launches")
    nvcc = product._nvcc()
    flags = product.ARCH + ["-std=c++17", "-I", product.INCLUDE, "-I", product.CSRC]

    def compile_one(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        subprocess.run([nvcc] + flags + ["-c", src, "-o", obj], check=True)
        return obj

    with ThreadPoolExecutor() as pool:
        objs = list(pool.map(compile_one, [os.path.join(product.CSRC, f) for f in SOURCES] + [NATIVE]))
    exe = str(out / "select_launches")
    # the shared runtime: the program's own definitions go before it
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc) or nvcc))),
                       "lib64")
    subprocess.run([nvcc, "-cudart", "shared", "-o", exe] + objs +
                   ["-Xlinker", "-rpath," + lib], check=True)
    text = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return [line.split() for line in text.splitlines()]


def test_no_call_lowers_a_kernels_limit_of_shared_memory(lines):
    """A kernel's limit is one for all threads of a process: a call that set its own size could
    lower it between another thread's limit and launch.  Every limit of a kernel is the same one,
    within the SM's, and every launch within it."""
    limits, asked = {}, {}
    for kind, kernel, *rest in lines:
        if kind == "limit":
            limits.setdefault(kernel, set()).add(int(rest[0]))
        elif kind == "launch":
            # (a launch within the default needs no limit, whatever other calls set)
            asked.setdefault(kernel, []).append(int(rest[2]))
    assert asked and limits
    for kernel, sizes in limits.items():
        assert len(sizes) == 1, "kernel %s: limits of %s bytes" % (kernel, sorted(sizes))
        assert max(sizes) <= MOST and max(asked[kernel]) <= min(sizes)
    for kernel in set(asked) - set(limits):
        assert max(asked[kernel]) <= DEFAULT_LIMIT
    assert all(rest[-1] == "0" for kind, *rest in lines if kind in ("select", "split"))


def splits(lines):
    """(head_dim, heads, items, tokens, partition, cluster or 0) of each split call."""
    cluster = 0
    for kind, *rest in lines:
        if kind == "launch":
            cluster, ctas = int(rest[4]), int(rest[1])
        elif kind == "split":
            dim, heads, items, tokens, partition, taken, _ = map(int, rest)
            if taken:
                assert ctas == items * cluster
            yield dim, heads, items, tokens, partition, cluster if taken else 0


def test_a_split_has_no_more_clusters_than_the_gpu_holds(lines):
    """36 of eight CTAs, 74 of four (two CTAs an SM; a cluster lies in one GPC): a wave of a few
    more would take as long again."""
    seen = set()
    for dim, heads, items, _, _, cluster in splits(lines):
        assert cluster in (0, 8 if items <= 36 else 4) or (dim, items, cluster) == (64, 37, 8)
        assert items <= 74 or cluster == 0
        assert heads <= 8 or cluster == 0
        seen.add((items, cluster))
    assert {(1, 8), (36, 8), (37, 4), (74, 4), (76, 0)} <= seen


def test_a_split_leaves_long_contexts_of_few_heads_to_a_plan(lines):
    """A warp of a cluster has 64 KB of keys and values at most (128 KB of more than four query
    heads with eight CTAs), or half of what the plan's partitions would give a warp."""
    for dim, heads, items, tokens, partition, cluster in splits(lines):
        if heads > 8 or items > 74:
            continue
        ways = 8 if items <= 36 or (dim == 64 and items == 37) else 4
        each = -(-tokens // (4 * ways))
        short = partition <= 512 and -(-tokens // partition) >= 16  # a partition is a warp's
        planned = partition if short else partition // 4
        small = each * dim * 4 <= (131072 if heads > 4 and ways == 8 else 65536)
        assert (cluster > 0) == (each <= 256 and (small or 2 * each <= planned)), (
            dim, heads, items, tokens, partition)
