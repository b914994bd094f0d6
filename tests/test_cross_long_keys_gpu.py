"""Cross attention over split keys where every block of 64 keys shows: random values
average out over a million keys, and a block that were left out or taken twice would not
be seen.  Here one key of each block stands out, with a value in a dim of its own.

Block b's key scores 30 against queries of group b % D and 0 against the others', as all
other keys do; its value is 1 in dim (b // D) % D, all others are 0.  A row of group g has
the n_g keys of its group at equal weights, so that dim d holds (its keys there) / n_g,
and a block more or less changes that by at least 1 / 4 here.

Tolerance.  The scores are exact and alike, the weights of the group are one number for
all, and 10^6 e^-30 < 2^-23 goes to the other keys.  The scaled maximum is rounded (2^-24 of
44, in log2 units: below 2^-18), in each chunk, and the joins add 2^-20: together below 2^-16
of the value and of the lse's units, whose own rounding is 2^-24 of 38 and so below 2^-18.
The output is rounded to bf16: 2^-8 of the value.  Of the other groups at most 5 D <= 640 keys hold
a 1 in a dim: 640 e^-30 < 2^-33.
"""
import numpy as np
import pytest
import torch

BLOCK, HIGH, SCALE = 64, 30.0, 0.125


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def counts(kv, Hkv, D, left_out=None, moved=0):
    """[Hkv, group, dim]: keys of the group whose value is 1 there; left_out: without that block; moved: with V that
    many blocks off."""
    b = torch.arange(-(-kv // BLOCK))
    if left_out is not None:
        b = b[b != left_out]
    out = torch.zeros(Hkv, D, D, dtype=torch.float64)
    for h in range(Hkv):
        c = (b + moved).clamp(max=-(-kv // BLOCK) - 1)
        out[h].view(-1).index_add_(0, (b + 7 * h) % D * D + (c // D) % D, torch.ones(len(b), dtype=torch.float64))
    return out


def expected(n, kv):
    """Rows of each group, and their lse, from the counts."""
    mine = n.sum(-1, keepdim=True)
    total = mine + (kv - mine) * np.exp(-HIGH)
    return n / total, HIGH + torch.log(total[..., 0])


def close(out, lse, want, want_lse):
    return bool(((out - want).abs() <= (2.0 ** -8 + 2.0 ** -15) * want + 2.0 ** -33).all()
                and ((lse - want_lse).abs() <= 2.0 ** -15).all())


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,qo,kv", [
    (8, 1, 64, 1, 1000003), (8, 1, 64, 4, 400001), (2, 2, 64, 12, 300001), (8, 2, 64, 3, 70001), (64, 4, 128, 1, 70001),
    (5, 1, 128, 4, 200003), (2, 1, 128, 150, 200003), (48, 1, 64, 3, 150001), (2, 1, 64, 300, 500009), (12, 4, 128, 20, 40000)])
@pytest.mark.parametrize("at", ["first", "last", "anywhere"])
def test_every_block_counts_once(Hq, Hkv, D, qo, kv, at):
    blocks = -(-kv // BLOCK)
    b = torch.arange(blocks, device="cuda")
    place = {"first": torch.zeros_like(b), "last": torch.full_like(b, BLOCK - 1),
             "anywhere": torch.randint(0, BLOCK, (blocks,), device="cuda", generator=torch.Generator("cuda").manual_seed(kv))}[at]
    pos = (b * BLOCK + place).clamp(max=kv - 1)
    k, v = (torch.zeros(kv, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for h in range(Hkv):
        k[pos, h, (b + 7 * h) % D] = HIGH
        v[pos, h, (b // D) % D] = 1.0
    plan = binding().CrossPlan([0, qo], [0], [kv], kv, Hq, Hkv, D, sm_scale=SCALE)
    assert plan.info()["num_decode_partials"] > 0
    want, want_lse = (t.cuda() for t in expected(counts(kv, Hkv, D), kv))
    G = Hq // Hkv
    head = torch.arange(Hq, device="cuda")
    for shift in range(0, D, qo * G):                     # until every group had its row
        group = (torch.arange(qo, device="cuda")[:, None] * G + head % G + shift) % D
        q = torch.zeros(qo, Hq, D, dtype=torch.bfloat16, device="cuda")
        q.scatter_(2, group[..., None], 8.0)
        out, lse = plan.attend(q, k, v, lse=torch.empty(qo, Hq, device="cuda"))
        assert close(out.double(), lse.double(), want[head // G, group], want_lse[head // G, group])
    assert plan.device_error() == 0


@pytest.mark.parametrize("Hkv,D,kv", [(1, 64, 1000003), (4, 128, 70001), (1, 128, 200003), (2, 64, 300001), (1, 64, 500009)])
def test_a_block_left_out_or_moved_would_show(Hkv, D, kv):
    """Mistakes planted in the expected values (CPU)."""
    want = expected(counts(kv, Hkv, D), kv)
    assert close(*want, *want) and not close(torch.zeros_like(want[0]), want[1], *want)
    blocks = -(-kv // BLOCK)
    for block in (0, 1, blocks // 2, blocks - 1):
        short = expected(counts(kv, Hkv, D, left_out=block), kv)
        assert not close(short[0], want[1], *want) and not close(want[0], short[1], *want)
    assert not close(expected(counts(kv, Hkv, D, moved=1), kv)[0], want[1], *want)
