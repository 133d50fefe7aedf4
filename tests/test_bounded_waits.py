"""What the attention kernels do when a bounded wait gives up, shown on their
sources: the path itself cannot be taken without a kernel that is broken on
purpose.

The block's give-up flag changes while its warps read it.  Lanes that take a
branch on their own reading part ways, and the votes, elections and barriers
of whole warps behind it wait for lanes that never come; and a producer that
goes on counting tiles it no longer copies waits for the wrong phases at its
end, so that the block can leave with copies in flight.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q4_weight_matmul_gb300", "csrc")
# what may touch the flag itself: its place, its start, a wait's own report (no warp-wide instruction depends on it)
PLAIN = (r"volatile int\* gave_up = ", r"^\s*\*gave_up = [01];$",
         r"^\s*if \(!tc::mbar_wait\(bar, [a-z &1]+, gave_up\) && !\*gave_up\) \{$")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["paged_attn_chunk.cuh", "paged_attn_few.cuh"])
def test_warps_decide_on_the_give_up_flag_together(name):
    lines = [line for line in source(name).splitlines() if "*gave_up" in line.replace("int* gave_up", "*gave_up")]
    stray = [line for line in lines if not any(re.search(p, line) for p in PLAIN)]
    assert not stray, stray
    vote = re.search(r"bool given_up\(volatile int\* gave_up\) \{ return __any_sync\(0xffffffffu, (.*)\); \}",
                     source("paged_attn_common.cuh"))
    assert vote and vote[1] == "*gave_up != 0"


@pytest.mark.parametrize("name,count", [("paged_attn_chunk.cuh", "n"), ("paged_attn_few.cuh", "issued")])
def test_a_producer_counts_only_what_it_copies_and_waits_for_it(name, count):
    text = source(name)
    stop, expect = text.index("if ((stop = given_up(gave_up))) break;"), text.index("tc::mbar_arrive_expect_tx(&full[slot]")
    assert text.count("mbar_arrive_expect_tx") == 1 and 0 < expect - stop < 120       # directly before a tile's first copy
    end = text.index("while (!stop && w.next(P, R, group));")
    assert expect < end
    drain = re.search(r"if \(lane == 0\) \{\s*for \(uint32_t j = %s < (\S+) \? 0 : %s - \1; j < %s; \+\+j\)\s*"
                      r"if \(!tc::mbar_wait_sleep\(&full\[j %% \1\], \(j / \1\) & 1\)\) break;" % (count, count, count), text[end:])
    assert drain, "the producer leaves without waiting for its last copies"
