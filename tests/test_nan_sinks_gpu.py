"""A sink of NaN: its head's rows are NaN in every kernel, and no other head's rows change."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)


def sinks_of(Hq, bad):
    s = torch.linspace(-1.0, 2.0, Hq, device="cuda")
    t = s.clone()
    t[bad] = float("nan")
    return s, t


def check(clean, out, bad, lse=None, clean_lse=None):
    keep = [h for h in range(out.shape[1]) if h != bad]
    assert bool(torch.isnan(out[:, bad]).all()) and torch.equal(out[:, keep], clean[:, keep])
    if lse is not None:
        assert bool(torch.isnan(lse[:, bad]).all()) and torch.equal(lse[:, keep], clean_lse[:, keep])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qo,kv,sms,items,split", [
    (2, 300, 0, False, False), (2, 20000, 0, False, True), (150, 100, 1, True, False), (150, 700, 1, True, False),
    (150, 2000, 8, True, True), (3, 0, 0, False, False)])
def test_cross(D, qo, kv, sms, items, split):
    g = torch.Generator(device="cuda").manual_seed(kv)
    q, k, v = randn(g, qo, 6, D), randn(g, kv, 2, D), randn(g, kv, 2, D)
    plan = binding().CrossPlan([0, qo], [0], [kv], kv, 6, 2, D, num_sms=sms)
    info = plan.info()
    assert (info["num_prefill_items"] > 0) == items and (info["num_decode_partials"] > 0) == split
    for bad in (0, 4):
        clean, nan = sinks_of(6, bad)
        a, la = plan.attend(q, k, v, clean, lse=torch.empty(qo, 6, device="cuda"))
        b, lb = plan.attend(q, k, v, nan, lse=torch.empty(qo, 6, device="cuda"))
        check(a, b, bad, lb, la)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("qo,kv", [(40, 40), (200, 513)])
def test_prefill(D, causal, qo, kv):
    g = torch.Generator(device="cuda").manual_seed(kv)
    Hq, Hkv, P = 4, 2, 16
    q, k, v = randn(g, qo, Hq, D), randn(g, kv, Hkv, D), randn(g, kv, Hkv, D)
    n = (kv + P - 1) // P
    pool = torch.zeros(n, 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(kv, device="cuda")
    pool[at // P, 0, :, at % P], pool[at // P, 1, :, at % P] = k, v
    table = torch.arange(n, dtype=torch.int32, device="cuda")
    ragged = binding().RaggedPlan([0, qo], [0, kv], Hq, Hkv, D, causal=causal)
    paged = binding().Plan([0, qo], [0, n], table, [kv - (n - 1) * P], Hq, Hkv, D, P, causal=causal, num_pages=n)
    for bad in (1, 2):
        clean, nan = sinks_of(Hq, bad)
        check(ragged.prefill(q, k, v, clean)[0], ragged.prefill(q, k, v, nan)[0], bad)
        check(paged.prefill(q, pool, clean)[0], paged.prefill(q, pool, nan)[0], bad)
        step = binding().Plan([0, 1], [0, n], table, [kv - (n - 1) * P], Hq, Hkv, D, P, num_pages=n)
        check(step.decode(q[:1], pool, clean)[0], step.decode(q[:1], pool, nan)[0], bad)
