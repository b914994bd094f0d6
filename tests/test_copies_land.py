"""A CTA must not end before the copies into its shared memory have landed, whichever
of its warps gave up a wait.  In decode.cu a warp waits for its own copies; elsewhere one
warp loads for others, which may give up while it has long issued its last copy.  No
wait can be made to run out on a sound kernel, so this reads the sources: every ring is
awaited with ptx::await_copies, under no condition on how the loading warp's own loop
ended: at that warp's end or, in prefill.cu, behind the CTA's last barrier where any
warp has set the flag that it gave up (CPU)."""
import os
import re

import pytest

from test_dependent_launch import CSRC, code

# Per file: the rings' (full barriers, stages, copies issued), in order.
RINGS = {
    "prefill.cu": ["B.k_full, C::kStagesK, issued_s[0]", "B.v_full, C::kStagesV, issued_s[1]",
                   "B.q_full, C::kQBufs, issued_s[2]"],
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
        # (4-bit keys are not copied by TMA)
        assert before.endswith((";", "}", "if (!kFour)", "if (warp == 0 && *abort_flag) {")), before[-40:]


def test_whoever_gives_up_in_prefill_says_so():
    """Every warp's failure goes through the flag, and the barrier lies between it and the waits."""
    source = code(os.path.join(CSRC, "prefill.cu"))
    assert re.search(r"auto fail = \[&\]\(int code\) \{\s*atomicOr\(a\.err, code\);\s*\*abort_flag = 1;\s*\};", source)
    assert source.count("ATTN_DEVICE_ERR_TIMEOUT") == source.count("fail(ATTN_DEVICE_ERR_TIMEOUT)") == 5
    assert re.search(r"__syncthreads\(\);\s*if \(warp == 0 && \*abort_flag\) \{\s*ptx::await_copies", source)
