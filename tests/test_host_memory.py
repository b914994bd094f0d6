"""Host memory that runs out while a plan is built is a status, as every other
failure of a C entry point, and not an exception that ends the process (CPU; in
a child process whose address space is limited)."""
import os
import subprocess
import sys

import pytest

from paged_kv_attention_sink_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, resource, sys
import numpy as np
lib = ctypes.CDLL(sys.argv[1])
rows = 1 << 27                                      # 1 GB of append slots
ind, pages, last = (np.array(a, dtype=np.int32) for a in ([0, rows], [0, rows // 16], [16]))
h, ws = ctypes.c_void_p(), ctypes.c_size_t()
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (128 << 20),) * 2)
P = ctypes.c_void_p(0x10000)
paged = lib.attn_plan(ind.ctypes.data_as(ctypes.c_void_p), pages.ctypes.data_as(ctypes.c_void_p), P,
                      last.ctypes.data_as(ctypes.c_void_p), 1, 1, 1, 64, 16, 1, ctypes.c_float(0.125), 1 << 24, 152,
                      ctypes.byref(h), ctypes.byref(ws))
print("status", paged, h.value)
"""


@pytest.mark.skipif(not os.path.exists(build.LIB) or not os.path.exists("/proc/self/statm"), reason="needs libattn.so and /proc")
def test_plan_without_memory():
    r = subprocess.run([sys.executable, "-c", CHILD, build.LIB], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split() == ["status", "1", "None"]     # ATTN_ERR_INVALID_ARG, nothing written
