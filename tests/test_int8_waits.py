"""The bounded waits of attend_int8's prompts, by the source: what happens once a wait has run out.  (A wait that runs out on
purpose is tested by tq_check_wait_expiry; these wait for other warps and the tensor core, which always answer.)"""
import re

from test_paged_waits import block, source


def test_every_wait_is_bounded_and_ends_its_role():
    t = source("tq_int8_prompt.cu")
    assert "try_wait" not in t and "test_wait" not in t                       # only through the library's bounded wait
    waits = re.findall(r"wait_parity_bounded\(([^;]*)\);", t)
    assert len(waits) == 2 and all("kFaultAttendWait" in w for w in waits)
    assert re.search(r"if \(!lost\) lost = !wait_parity_bounded\(bar, parity & 1, kFaultAttendWait\)", t)
    # a warp's lanes stay together: the votes and exchanges behind a wait need them all
    assert re.findall(r"\bwait\(([^)]*)\)", t) == ["bar, parity"] and "lost = __any_sync(0xffffffffu, lost)" in block(t, "auto wait_all")
    # each role's loop over tiles stops, and none waits for other threads in between but at the end
    assert t.count("for (int i = 0; i < n && !lost; ++i)") == 3
    assert "bar.sync" not in t and len(re.findall(r"__syncthreads\(\)", t)) == 2


def test_what_was_not_computed_is_nan():
    t = source("tq_int8_prompt.cu")
    assert re.search(r"const float f = lost \? nan", t) and re.search(r"lost \? nan : sum", t)
    # products in flight end before the tensor memory is freed
    assert t.index("commit_to(drained)") < t.index("wait_parity_bounded(drained") < t.index("tcgen05.dealloc")


def test_registers_dealt_out_fit_the_block():
    """setmaxnreg draws on what the block was launched with: 512 threads of 128."""
    t = source("tq_int8_prompt.cu")
    of = {k: [int(x) for x in re.findall(rf"setmaxnreg\.{k}\.sync\.aligned\.u32 (\d+)", t)] for k in ("inc", "dec")}
    assert len(of["inc"]) == 1 and len(of["dec"]) == 2
    assert 256 * of["inc"][0] + 128 * sum(of["dec"]) <= 512 * 128
    assert "kWarps = 16" in t


def test_fault_bit():
    assert "kFaultAttendWait = 128u" in source("tq_int8_prompt.cu")
    import os
    from conftest import ROOT
    with open(os.path.join(ROOT, "include", "tq.h")) as f:
        assert "128 = a wait of tq_attend_int8" in f.read()
