"""The bounded waits of the paged append, by its source: what a warp does once a wait of its own
has run out.  (A wait that runs out on purpose is tested by tq_check_wait_expiry; the append's
wait for the tensor core, which always answers.)"""
import os
import re

from conftest import ROOT


def source(name):
    with open(os.path.join(ROOT, "compressed_kv_cache_gb300", "csrc", name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, start):
    """The braces that follow `start`."""
    i = text.index("{", text.index(start))
    depth = 0
    for j in range(i, len(text)):
        depth += (text[j] == "{") - (text[j] == "}")
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError(start)


def test_a_lost_warp_takes_no_further_part():
    t = source("tq_append.cu")
    assert re.search(r"lost = __any_sync\(0xffffffffu, !wait_parity_bounded\(", t)      # the whole warp's
    make = block(t, "auto make_operand")
    assert re.match(r"\{\s*if \(lost\) \{\s*ahead\.next\(a\.tiles\);\s*return;\s*\}", make)
    issue = block(t, "auto issue_tile")
    assert issue.index("wait(whole_op") < issue.index("if (lane == 0 && !lost)") < issue.index("tcgen05.commit")
    assert issue.index("if (lane == 0 && !lost)") < issue.index("mma_f16")
    assert re.search(r"if \(!lost\) \{[^}]*search_tile", block(t, "while (now.item < last)"), re.S)


def test_fault_bits_of_the_paged_calls_have_one_meaning_each():
    """32: a number out of range; 64: a wait that ran out.  A shared-memory layout that the decode
    is not built for is refused by the host."""
    for name in sorted(os.listdir(os.path.join(ROOT, "compressed_kv_cache_gb300", "csrc"))):
        t = source(name)
        assert not re.search(r"wait_parity_bounded\([^;]*kFaultPaged\)", t), name
    assert "kFaultPagedWait = 64u" in source("tq_paged.cuh")
    assert "kFaultPagedWait" in source("tq_append.cu")
    kernel = block(source("tq_paged_split.cuh"), "paged_split_kernel")
    assert "return;" not in kernel and kernel.count("kFaultPaged") == 1
    launch = block(source("tq_paged_split.cuh"), "cudaError_t launch_one")
    assert launch.index("kept > kFirst") < launch.index("cudaLaunchKernelEx")
    with open(os.path.join(ROOT, "include", "tq.h")) as f:
        assert "64 = a wait of" in f.read()
