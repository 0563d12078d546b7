"""Order of barriers in the scan of the scalar-gate delta rule, read from its source (a race need not show in any run).

In the forward the two chain waves store over each other's values of a chunk (the second terms of Y) before the
step's barrier A.  Both must have read those values behind a barrier that the other one passes before its
store: barrier B of the step before, and for chunk 0 one of the opening barriers."""
import os
import re

import gated_delta_rule_45_amd as kda

SOURCE = os.path.join(os.path.dirname(kda.__file__), "csrc", "kda_gdn_scan.h")
BARRIER = "__syncthreads()"


def chain_waves():
    """The code of the chain waves without comments: what stands before the loop over the steps, and the loop."""
    text = open(SOURCE).read()
    text = text[text.index("- chain waves\n"):]
    text = re.sub(r"//[^\n]*", "", text)
    head, loop = text.split("for (int s = 0; s < nch; ++s) {", 1)
    return head, loop[:loop.index("const bool part")]


def test_values_are_read_a_barrier_before_they_are_stored_over():
    head, loop = chain_waves()
    store = loop.index("hand_put<BF>(V")
    assert BARRIER not in loop[:store]  # so a read without a barrier behind it would meet the other wave's store
    first = head.index("fetch(0)")
    assert BARRIER in head[:first], "chunk 0 is in LDS behind the first opening barrier"
    assert BARRIER in head[first:], "no barrier between the read of chunk 0's values and the first step's store"
    ahead = loop.index("fetch(s + 1)")
    assert BARRIER in loop[ahead:], "no barrier between the read of a chunk's values and its step's store"


def test_every_group_of_waves_meets_the_same_barriers():
    """Three opening barriers and two in a step, in every branch of the kernel (a wave that misses one hangs the others)."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read().replace("// ------", "GROUP"))
    groups = text[text.index("GROUP"):].split("GROUP")[1:]
    assert len(groups) == 5
    for g in groups:
        head, loop = g.split("for (int s = 0; s < nch; ++s) {", 1)
        chain = "- chain waves" in head
        if "const bool part" in loop:
            loop = loop[:loop.index("const bool part")]
        # the chain's barrier A stands in the forward's and in the reverse branch, of which a step takes one
        assert head.count(BARRIER) == 3 and loop.count(BARRIER) == (3 if chain else 2), head[:80]
