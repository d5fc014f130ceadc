"""CPU: what the decode entry points hand to the work plan and to the attention
kernels.  native/plan_params.cpp compiles them as they are over stand-ins for the
launches, and calls them on a stack filled with one pattern after another."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from paged_kv_cache_312_gb300 import build as product

NATIVE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "plan_params.cpp")
FIELDS = ("rc spare slots max_groups partition cta_parts stage counters parts grid planned").split()


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """{call: [fields for each pattern on the stack]}."""
    out = tmp_path_factory.mktemp("plan")
    nvcc = product._nvcc()
    flags = product.ARCH + ["-std=c++17", "-I", product.INCLUDE, "-I", product.CSRC]

    def compile_one(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        subprocess.run([nvcc] + flags + ["-c", src, "-o", obj], check=True)
        return obj

    sources = [os.path.join(product.CSRC, f) for f in ("api.cu", "api_q4.cu")] + [NATIVE]
    with ThreadPoolExecutor() as pool:
        objs = list(pool.map(compile_one, sources))
    exe = str(out / "plan_params")
    # the shared runtime: the program's own definitions go before it
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(nvcc) or nvcc))),
                       "lib64")
    subprocess.run([nvcc, "-cudart", "shared", "-o", exe] + objs +
                   ["-Xlinker", "-rpath," + lib], check=True)
    text = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    calls = {}
    for line in text.splitlines():
        name, _, *values = line.split()
        calls.setdefault(name, []).append(dict(zip(FIELDS, map(int, values))))
    return calls


def test_no_field_of_a_plan_comes_from_the_stack(launches):
    for name, seen in launches.items():
        assert all(s == seen[0] for s in seen), (name, seen)


@pytest.mark.parametrize("name", ["split-warp-partitions", "split-many", "unsplit", "wide-group"])
def test_16_bit_plans_have_no_spare_records(launches, name):
    """`spare` is for launches whose grid has that many records beyond one a row;
    the 16-bit launches' grids hold max_groups records a row and no more."""
    for s in launches[name]:
        assert s["rc"] == 0 and s["planned"] == 1 and s["spare"] == 0


def test_a_4_bit_split_call_has_room_for_its_spare_records(launches):
    rows = 64 * 8
    for s in launches["q4-split"]:
        assert s["planned"] == 1 and s["spare"] == 2 * s["slots"] > 0
        assert s["grid"] == min(rows * s["parts"], rows + s["spare"])


@pytest.mark.parametrize("name", ["huge-partition", "q4-huge-partition"])
def test_a_partition_beyond_every_context_is_one_a_context(launches, name):
    """2^31 - 32 tokens a partition, where context plus partition passes 31 bits."""
    for s in launches[name]:
        assert s["rc"] == 0 and s["parts"] == 1 and s["grid"] == 4 * 8
