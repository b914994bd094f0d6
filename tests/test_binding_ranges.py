"""Host numbers that 32 bits do not hold are refused by the binding, not wrapped into others (CPU)."""
import numpy as np
import pytest
import torch

FAR = 1 << 32


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


@pytest.mark.parametrize("far", [FAR, -FAR, FAR + 3, (1 << 31), -(1 << 31) - 1])
@pytest.mark.parametrize("kind", [list, np.array, torch.tensor])
def test_plans(far, kind):
    b = binding()
    ok = dict(qo_indptr=[0, 1], kv_start=[0], kv_len=[5])
    for name in ok:
        args = {**ok, name: ok[name][:-1] + [far]}
        with pytest.raises(ValueError):
            b.CrossPlan(*(kind(x) for x in args.values()), 5, 8, 2, 64, num_sms=8)
    table = torch.zeros(1, dtype=torch.int32)
    for qo, kv, last in (([0, far], [0, 1], [5]), ([0, 1], [0, far], [5]), ([0, 1], [0, 1], [far])):
        with pytest.raises(ValueError):
            b.Plan(kind(qo), kind(kv), table, kind(last), 8, 2, 64, 16, num_pages=1, num_sms=8)
    for qo, kv in (([0, far], [0, 5]), ([0, 1], [0, far])):
        with pytest.raises(ValueError):
            b.RaggedPlan(kind(qo), kind(kv), 8, 2, 64, num_sms=8)
    with pytest.raises(ValueError):
        b.Rope([0.5] * 8, axis=kind([0] * 7 + [far]))


def test_sizes():
    b = binding()
    for page_size in (0, -1, 1 << 31, FAR + 16):
        with pytest.raises(ValueError):
            b.PagePool([torch.zeros(4, 16)], page_size)
    for kv_rows in (-1, 1 << 31, FAR + 5):
        with pytest.raises(ValueError):
            b.CrossPlan([0, 1], [0], [5], kv_rows, 8, 2, 64, num_sms=8)


def test_what_fits_is_taken():
    for x in ([0, -1, (1 << 31) - 1, -1 << 31], np.array([3], np.int64), np.array([7], np.uint8), torch.tensor([2, 5]), []):
        assert binding()._i32_host(x).tolist() == [int(v) for v in x]
    assert binding().Rope([0.5] * 8, axis=np.arange(8) % 3).n_axes == 3
