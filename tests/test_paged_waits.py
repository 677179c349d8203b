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
