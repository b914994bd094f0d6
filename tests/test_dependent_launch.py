"""Kernels that are launched as programmatic dependents are resident while the
kernel before them still writes what they will read.  The read-only data path
(__ldg, ld.global.nc, const __restrict__ parameters) promises data that does
not change for as long as the kernel runs, so none of them may use it; this
reads their sources for it (CPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_attention_sink_gb300", "csrc")


def code(path):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def dependent_sources():
    """The files that launch dependents, and the headers of device code that they include."""
    found = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_dependent(" in code(p)]
    headers = {os.path.join(CSRC, h) for p in found for h in re.findall(r'#include "(\w+\.cuh)"', code(p))}
    return sorted(os.path.basename(p) for p in {*found, *headers})


def test_dependents_are_found():
    assert {"kv4.cu", "decode4.cu", "evict.cu", "keyweights.cu", "kv4_stage.cuh", "ptx.cuh"} <= set(dependent_sources())


@pytest.mark.parametrize("name", dependent_sources())
def test_dependents_take_no_read_only_loads(name):
    source = code(os.path.join(CSRC, name))
    assert re.findall(r"__ldg\w*|__restrict__|ld\.global\S*\.nc\S*|__constant__", source) == []
