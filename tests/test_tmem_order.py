"""tcgen05.alloc waits without a limit until another block of the SM gives its columns
back.  A kernel that held them while it waited for the kernels before it on the stream,
one of which wanted them on the same SM, would wait for good, and so would one whose
next kernel took them first.  No test could show that without hanging a GPU: the order
is read from the sources, in every kernel that allocates."""

import glob
import os
import re

import pytest

from routed_moe_layer_b200 import build


def kernels():
    """(file, name, body) of every kernel that allocates tensor memory; the body ends where
    the kernel's function does (a closing brace in the first column)."""
    found = []
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__.*?\b(\w+_kernel)\s*\(.*?\n}", text, re.S):
            if "tmem_alloc" in m.group(0):
                found.append((os.path.basename(path), m.group(1), m.group(0)))
    return found


def test_all_are_found():
    assert {name for _, name, _ in kernels()} == {
        "grouped_gemm_kernel", "grouped_gemm_swap_kernel", "grouped_gemm_swap_fp8_kernel",
        "swap_fused_kernel", "grouped_mx_kernel", "grouped_mx_few_kernel", "router_gemm_kernel"}


@pytest.mark.parametrize("file,name,body", kernels(), ids=lambda v: v if len(v) < 40 else "")
def test_tensor_memory_is_taken_behind_the_wait(file, name, body):
    alloc = body.index("tmem_alloc")
    waits = [m.start() for m in re.finditer(r"(if \((!?early)\) )?pdl_wait\(\);", body)
             if m.start() < alloc]
    # one wait of all threads, or one where the kernel is early and one where it is not
    last = [re.match(r"(if \(!?early\) )?", body[w:]).group(0) for w in waits]
    assert "" in last or {"if (early) ", "if (!early) "} <= set(last), (file, name)
    if "early" in body:  # other warps' waits do not count: that of the allocating warp is the last
        assert re.search(r"if \(early\) pdl_wait\(\);\s*tmem_alloc\(", body)
        # and the next kernel starts after it
        assert body.index("pdl_launch_dependents") > alloc
