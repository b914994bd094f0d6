"""Kernels that run beside the launch before them (kernels.h): only those of a cross
attention call do, behind a kernel that waits before it lets them start, and each
waits before it ends.  Read from the sources (CPU)."""
import glob
import os
import re

from test_dependent_launch import CSRC, code

WAIT, GO = "ptx::grid_dependency_wait();", "ptx::grid_dependents_go();"


def test_only_cross_attention_launches_late_kernels():
    late = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if re.search(r"\.late\b", code(p))}
    assert late == {"cross.cu", "prefill.cu"}


def test_the_first_kernel_waits_before_it_opens():
    source = code(os.path.join(CSRC, "cross.cu"))
    wait, open_ = source.index(f"if (!a.late) {WAIT}"), source.index(f"if (a.open) {GO}")
    assert wait < open_ and GO not in source[:open_]
    launch = source[source.index("attn_status launch_cross"):]
    assert launch.index("a.late = a.open = 0;") < launch.index("a.open =") < launch.index("a.late = 1;")


def test_late_kernels_wait_before_they_end():
    """No return between a late kernel's start and its wait."""
    for name, kernel in (("cross.cu", "cross_few_kernel"), ("prefill.cu", "prefill_sink_attn_kernel")):
        source = code(os.path.join(CSRC, name))
        body = source[re.search(rf"^{kernel}\(", source, re.M).start():]
        end = body.index(f"a.late) {WAIT}", body.index(f"!a.late) {WAIT}") + 20)
        head = re.sub(r"auto \w+ = \[&\].*?\n        \};", "", body[:end], flags=re.S)     # (lambdas return to the kernel)
        assert not re.search(r"\breturn\b", head), re.search(r".*\breturn\b.*", head).group(0)
