"""What the routed experts' kernels do when a bounded wait gives up, shown on
their sources: the path itself cannot be taken without a kernel that is broken
on purpose.  Warps decide together, and whoever copies waits for its copies
before it leaves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q4_weight_matmul_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_a_wait_is_bounded_and_a_warp_agrees_on_it():
    text = source("moe.cuh")
    agreed = text[text.index("bool agreed("):text.index("bool warp_wait(")]
    assert agreed.index("if (__all_sync(~0u, ok)) return true;") < agreed.index("*gave_up = 1;") < agreed.index("return false;")
    wait = text[text.index("bool warp_wait("):]
    wait = wait[:wait.index("\n}\n")]
    loop = wait[wait.index("while ("):]
    assert "__all_sync" in loop and "agreed(!*gave_up && " in loop and "kTimeoutCycles" in loop and "return false;" in loop


@pytest.mark.parametrize("name", ["moe_few.cuh", "moe_many.cuh"])
def test_warps_wait_together(name):
    """No wait but the warps' own, one lane's for its own copies at the end, and the one for the last products."""
    lines = source(name).splitlines()
    waits = [line for line in lines if re.search(r"mbar_wait\w*\(|mbar_try_wait\(", line) and "warp_wait" not in line]
    plain = r"^\s*if \(!tc::mbar_wait_sleep\(&[SH]\.(\w+)\[.*\], .*\)\) (break|atomicOr\(err, 1\));$"
    polls = [line for line in waits if not re.match(plain, line)]
    assert all("ok = tc::mbar_try_wait" in line or "while (!(ok" in line for line in polls), polls
    for i, line in enumerate(lines):                                   # the flag is read in a vote's argument alone
        if "*gave_up" in line.replace("int* gave_up", "") and not re.match(r"^\s*\*gave_up = [01];$", line):
            assert "kTimeoutCycles" in line and "return agreed(ok, gave_up, err);" in "\n".join(lines[i:i + 8]), line


@pytest.mark.parametrize("name,copies", [("moe_few.cuh", {"full"}), ("moe_many.cuh", {"xfull", "sfull", "rfull"})])
def test_who_copies_waits_for_its_copies(name, copies):
    text = source(name)
    asked = set(re.findall(r"mbar_arrive_expect_tx\(&[SH]\.(\w+)\[", text))
    drained = {m for m in re.findall(r"mbar_wait_sleep\(&[SH]\.(\w+)\[", text)} - {"drain"}
    assert asked == copies == drained
    if name == "moe_few.cuh":
        last = text.rindex("copies_arrive(&H.full[slot]);")
        assert "cp.async.wait_all" in text[last:]
    else:                                                              # tensor memory goes when every product is done
        assert text.index("mma_commit(&S.drain[mt])") < text.index("mbar_wait_sleep(&S.drain[mt]") < text.index("tmem_dealloc")
