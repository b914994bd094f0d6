"""Cross attention after a wait that ran out (recorded by hand in the error word: no
wait of a sound kernel does): the states of split keys, which may then be an older
call's, are not joined, and once the error is read everything is written again."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT = 2


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def error_word(plan):
    """The plan's error word as a view of its workspace: the one word whose bit plan.device_error() returns."""
    words = plan.workspace[:plan.workspace.numel() // 4 * 4].view(torch.int32)
    for at in range(0, len(words), 64):                     # 256-byte aligned
        old = int(words[at])
        words[at] = old | 1 << 20
        code = plan.device_error()
        words[at] = old
        if code == 1 << 20:
            return words[at:at + 1]
    raise AssertionError("no error word in the workspace")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qo,kv,sms,split", [
    ([3, 2, 20], [20000, 10, 9000], 0, [0, 2]), ([150, 90, 1], [2000, 100, 40], 8, [0])])
def test_split_keys_are_not_joined(D, qo, kv, sms, split):
    g = torch.Generator(device="cuda").manual_seed(1)
    start = np.concatenate([[0], np.cumsum(kv)[:-1]])
    q, k, v = (torch.randn(n, h, D, device="cuda", generator=g).to(torch.bfloat16)
               for n, h in ((sum(qo), 6), (sum(kv), 2), (sum(kv), 2)))
    plan = binding().CrossPlan(np.concatenate([[0], np.cumsum(qo)]), start, kv, sum(kv), 6, 2, D, num_sms=sms)
    assert plan.info()["num_decode_partials"] > 0
    want, want_lse = plan.attend(q, k, v, lse=torch.empty(len(q), 6, device="cuda"))
    rows = np.concatenate([[0], np.cumsum(qo)])
    joined = torch.zeros(len(q), dtype=torch.bool, device="cuda")
    for b in split:
        joined[rows[b]:rows[b + 1]] = True
    word = error_word(plan)
    for code, left in ((0, 0), (TIMEOUT, int(joined.sum())), (0, 0)):
        word |= code
        out, lse = torch.full_like(q, float("nan")), torch.full((len(q), 6), float("nan"), device="cuda")
        plan.attend(q, k, v, out=out, lse=lse)
        blank = torch.isnan(out).all(-1).all(-1)
        assert int(blank.sum()) == left and (not left or torch.equal(blank, joined))
        assert torch.equal(out[~blank], want[~blank]) and torch.equal(lse[~blank], want_lse[~blank])
        assert bool(torch.isnan(lse[blank]).all())
        assert plan.device_error() == code and plan.device_error() == 0
