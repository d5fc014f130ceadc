"""CPU: a kernel that is launched as a programmatic dependent of the one before it
may be resident while that one runs, and sees its writes only after its own
griddepcontrol.wait.  Read from the source: what a kernel takes from memory before
the wait is nothing, or (the work plan) read again behind it."""
import glob
import os
import re

import pytest

from paged_kv_cache_312_gb300 import build as product

WAIT = re.compile(r"griddepcontrol\.wait|wait_for_previous\(\);")
# an element of an array among the kernel's parameters: p.array[i], *p.word, pp.array[i]
READ = re.compile(r"\bpp?\.\w+\s*\[|(?<![\w)\]] )\*\s*pp?\.\w+|__ld\w+\(\s*pp?\.\w+[^;]*")


def kernels():
    """(file, kernel, body) of every kernel that waits for the one before it."""
    for path in sorted(glob.glob(os.path.join(product.CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        parts = re.split(r"__global__\s+void", text)
        for part in parts[1:]:
            name = re.search(r"(\w+)\s*\(\s*const", re.sub(r"__launch_bounds__\(.*?\)\)?\)?\s",
                                                           "", part, flags=re.S))
            body = part[:part.index("\n}\n")]
            if WAIT.search(body):
                yield os.path.basename(path), name.group(1), body


def test_the_kernels_are_found():
    names = {name for _, name, _ in kernels()}
    assert {"decode_tc_kernel", "decode_plan_kernel", "decode_tc05_kernel", "decode_q4_kernel",
            "write_kernel", "read_kernel", "extend_small_kernel", "extend_rows_kernel",
            "release_small_kernel", "release_rows_kernel", "merge_q4_kernel"} <= names


@pytest.mark.parametrize("file,name,body", list(kernels()), ids=lambda x: x if len(x) < 40 else "")
def test_nothing_is_taken_from_memory_before_the_wait(file, name, body):
    at = WAIT.search(body).start()
    before = {re.sub(r"\s+", " ", m.group(0)) for m in READ.finditer(body[:at])}
    again = {re.sub(r"\s+", " ", m.group(0)) for m in READ.finditer(body[at:])}
    # read early through L2, and read again
    early = {x for x in before if x.startswith("__ldcg") and x in again}
    assert before <= early, (file, name, sorted(before - early))
