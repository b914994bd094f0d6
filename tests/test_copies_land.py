"""A CTA must not end before the copies into its shared memory have landed, whichever
of its warps gave up a wait.  In decode.cu a warp waits for its own copies; elsewhere one
warp loads for others, which may give up while it has long issued its last copy.  No
wait can be made to run out on a sound kernel, so this reads the sources: each loading
warp ends with ptx::await_copies over every ring that it fills, under no condition on
how its loop ended (CPU)."""
import os
import re

import pytest

from test_dependent_launch import CSRC, code

# Per file: the rings' (full barriers, stages, copies issued), in order.
RINGS = {
    "prefill.cu": ["full0, n_stages, issued", "B.q_full, C::kQBufs, q_issued"],
    "cross.cu": ["full, C::kStages, it"],
    "keyweights.cu": ["q_full, C::kStages, s", "k_full, 1, 1"],
}


def test_every_kernel_that_loads_for_other_warps_is_listed():
    loads = {f for f in os.listdir(CSRC) if f.endswith(".cu") and "tma_load" in code(os.path.join(CSRC, f))}
    assert loads == {*RINGS, "decode.cu"}


@pytest.mark.parametrize("name", RINGS)
def test_loading_warps_await_their_copies(name):
    source = code(os.path.join(CSRC, name))
    found = list(re.finditer(r"ptx::await_copies\(([^;]*)\);", source))
    assert [m.group(1) for m in found] == RINGS[name]
    for m in found:
        before = source[:m.start()].rstrip()
        assert before.endswith((";", "}", "if (!kFour)")), before[-40:]   # (4-bit keys are not copied by TMA)
