"""Rows whose first keys all score -inf: prefill (paged, ragged) and cross attention
against the plain 64-bit form.

Those keys weigh nothing, however many tiles they fill and whatever the scores
behind them are: of ordinary size, so far below 0 that exp underflows unless the
maximum is theirs, or rising from key to key.

Tolerance.  P is rounded to bf16, by at most 2^-8 of a weight, and O normalised by the
sum of that rounded P: (1 + 2^-8) / (1 - 2^-8) - 1 < 2^-7 + 2^-13 of sum w |v|.  The
output's own rounding is 2^-8 of the value.  Scores are fp32 sums of D products, scaled
once, with scale sum |q k| <= 500 here: 132 roundings of 2^-24 of 500 are below 2^-7,
relative in a weight and absolute in the lse (exponentials and joins add 2^-20).  Weights
below 2^-126 beside a sink's may be flushed to 0: 2,000 of them times |v| < 8 are below
2^-111.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 0.125
LOWEST = torch.finfo(torch.bfloat16).min


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def inputs(rows, keys, lead, Hq, Hkv, D, behind, lowest, seed):
    """q, k, v of one sequence whose first `lead` keys score -inf: by keys of -inf for every row, or (lowest) by
    the type's lowest value times 4, which passes fp32, for every third row alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(rows, Hq, D, device="cuda", generator=g)
    k = torch.randn(keys, Hkv, D, device="cuda", generator=g)
    v = torch.randn(keys, Hkv, D, device="cuda", generator=g)
    q[..., 0], k[..., 0], q[..., 1], k[..., 1] = 1.0, 0.0, 1.0, 0.0
    if lowest:
        q[..., 0] = 0.0
        q[::3, :, 0] = 4.0
    k[:lead, :, 0] = LOWEST if lowest else -float("inf")
    n = keys - lead
    if behind == "low":
        k[lead:, :, 1] = -3200.0                        # -400
    elif behind == "rising":
        k[lead:, :, 1] = torch.linspace(-2400.0, 2400.0, n, device="cuda")[:, None]   # -300 .. 300
    return tuple(t.to(torch.bfloat16) for t in (q, k, v))


def plain(q, k, v, sinks, causal):
    rows, Hq, keys = q.shape[0], q.shape[1], k.shape[0]
    kk, vv = (t.double().repeat_interleave(Hq // k.shape[1], 1) for t in (k, v))
    s = torch.einsum("rhd,thd->rht", q.double(), kk) * SCALE
    if causal:
        seen = torch.arange(keys, device="cuda")[None] <= torch.arange(rows, device="cuda")[:, None] + keys - rows
        s = torch.where(seen[:, None], s, -float("inf"))
    s = torch.where(s < -1e30, -float("inf"), s)        # (what passes fp32)
    z = s if sinks is None else torch.cat((s, sinks.double()[None, :, None].expand(rows, -1, 1)), -1)
    lse = torch.logsumexp(z, -1)
    w = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("rht,thd->rhd", w, vv), torch.einsum("rht,thd->rhd", w, vv.abs()), lse


def compare(out, lse, want, mag, want_lse):
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -13 + 2.0 ** -7) * mag + 2.0 ** -111
    assert bool(((out.double() - want).abs() <= tol).all())
    gone = torch.isinf(want_lse)
    assert torch.equal(lse.double()[gone], want_lse[gone])
    assert bool(((lse.double() - want_lse)[~gone].abs() <= 2.0 ** -7).all())


def sinks_of(kind, Hq):
    return {"none": None, "gone": torch.full((Hq,), -float("inf"), device="cuda"),
            "some": torch.linspace(-350.0, 3.0, Hq, device="cuda")}[kind]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sms", [1, 8])                 # whole keys; long ones split
@pytest.mark.parametrize("lead,keys", [(128, 129), (128, 700), (200, 1500), (300, 2000), (900, 1601)])
@pytest.mark.parametrize("behind", ["ordinary", "low", "rising"])
def test_cross(D, sms, lead, keys, behind):
    for lowest in (False, True):
        q, k, v = inputs(150, keys, lead, 6, 2, D, behind, lowest, seed=lead + keys)
        plan = binding().CrossPlan([0, len(q)], [0], [keys], keys, 6, 2, D, sm_scale=SCALE, num_sms=sms)
        info = plan.info()
        assert info["num_decode_units"] == 0 and (info["num_decode_partials"] > 0) == (sms > 1 and keys >= 1500)
        for kind in ("none", "gone", "some"):
            sinks = sinks_of(kind, 6)
            out, lse = plan.attend(q, k, v, sinks, lse=torch.empty(len(q), 6, device="cuda"))
            compare(out, lse, *plain(q, k, v, sinks, False))
        assert plan.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lead,keys,rows", [(128, 300, 300), (300, 900, 200), (129, 513, 513)])
@pytest.mark.parametrize("behind", ["ordinary", "low", "rising"])
def test_prefill(D, causal, lead, keys, rows, behind):
    Hq, Hkv, P = 4, 2, 16
    for lowest in (False, True):
        q, k, v = inputs(rows, keys, lead, Hq, Hkv, D, behind, lowest, seed=lead + keys)
        n_pages = (keys + P - 1) // P
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(keys))
        pool = torch.zeros(n_pages, 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
        page, row = order.cuda()[torch.arange(keys, device="cuda") // P], torch.arange(keys, device="cuda") % P
        pool[page, 0, :, row], pool[page, 1, :, row] = k, v
        ragged = binding().RaggedPlan([0, rows], [0, keys], Hq, Hkv, D, causal=causal, sm_scale=SCALE)
        paged = binding().Plan([0, rows], [0, n_pages], order.to(torch.int32).cuda(), [keys - (n_pages - 1) * P], Hq, Hkv, D,
                               P, causal=causal, sm_scale=SCALE, num_pages=n_pages)
        for kind in ("none", "gone", "some"):
            sinks = sinks_of(kind, Hq)
            want = plain(q, k, v, sinks, causal)
            out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
            ragged.prefill(q, k, v, sinks, out, lse)
            compare(out, lse, *want)
            out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
            paged.prefill(q, pool, sinks, out, lse)
            compare(out, lse, *want)
        assert paged.device_error() == 0 and ragged.device_error() == 0
