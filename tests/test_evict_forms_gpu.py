"""Eviction of rows that are read in chunks, in each form that reads them so: a
CTA with all of an SM (few rows), or with a part of it (many), which either
copies too (out of place) or leaves that to a second kernel (in place).  The
choice is computed here again, so that a case cannot slip to another form."""
import pytest
import torch

import test_evict_gpu

pytestmark = pytest.mark.gpu

CASES = [  # lengths, KV heads, budget, recent, form
    ([50001, 40], 1, 20011, 100, "few"),
    ([12003] + [17] * 89, 2, 5000, 7, "few"),                    # more rows than SMs, but one would not fit a part
    ([49152] + [17] * 79, 2, 40000, 0, "few"),
    ([49153] + [17] * 79, 2, 40000, 0, "many"),                  # does not fit a whole SM either
    ([12003] + [17] * 199, 2, 5000, 7, "many"),
    ([30001, 11265, 11264] + [33] * 317, 1, 11264, 11264, "many"),
]


def form(kv, Hkv):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, longest = len(kv) * Hkv, max(kv)
    return "few" if rows <= sms or (rows <= 2 * sms and 11 * 1024 < longest <= 48 * 1024) else "many"


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv,Hkv,budget,recent,want", CASES)
def test_rows_read_in_chunks(in_place, kv, Hkv, budget, recent, want):
    assert form(kv, Hkv) == want
    test_evict_gpu.test_evict_rows_longer_than_shared_memory(in_place, kv, Hkv, budget, recent)
