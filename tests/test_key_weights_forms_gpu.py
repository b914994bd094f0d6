"""Key weights of prefill rows in both forms of their kernel: few CTAs (or many
steps a tile) take the long one, many CTAs of few steps the short one.  Every
case names the form it is for, and the choice is computed here again, so that a
case cannot slip to the other one.  A plan for one SM makes a few CTAs many."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from helpers import make_plan, syn
from test_evict_gpu import pools, run_weights, some_lse
from test_kv4_gpu import batch_of, dev, dev_bf16

pytestmark = pytest.mark.gpu

SHORT_STEPS = 64


def steps_of(rows, G):
    heads = min(G, 128)
    return -(-rows // (128 // heads)) * -(-G // heads)


def forms(batch, window, num_sms):
    """The forms that the batch's requests take: [one] for all, or [of those of many steps, of the others]."""
    G, Hkv = batch.num_qo_heads // batch.num_kv_heads, batch.num_kv_heads
    req = [(int(n), -(-int(kv) // 128)) for n, kv in zip(batch.qo_lens, batch.kv_lens) if n > 1]
    many = [r for r in req if steps_of(r[0], G) > SHORT_STEPS]
    few = [r for r in req if steps_of(r[0], G) <= SHORT_STEPS]

    def load(req, window):
        per = [(steps_of(min(n, window) if window else n, G), t) for n, t in req]
        return sum(t for _, t in per), sum(s * t for s, t in per), max(s for s, _ in per)

    def short(req, window):
        tiles, steps, _ = load(req, window)
        ctas, per_sm = tiles * Hkv, 4 if batch.head_dim == 64 else 2
        return ctas > num_sms and steps <= SHORT_STEPS * tiles and 2 * steps * num_sms <= 3 * per_sm * ctas * tiles

    name = lambda req: "short" if short(req, window) else "long"
    _, steps, longest = load(req, 0)
    if many and few and short(req, 0) and 8 * longest * num_sms > 5 * steps * Hkv:
        return [name(many), name(few)]
    return [name(req)]


def check(batch, four, window, num_sms, want_forms, decay=0.75):
    _, pool, vals = pools(batch, four, seed=3)
    plan = make_plan(batch, dev(batch.page_table), num_sms=num_sms)
    assert forms(batch, window, num_sms) == want_forms
    lse = some_lse(batch, vals)
    prev = np.random.default_rng(5).exponential(size=(batch.num_pages, batch.num_kv_heads, batch.page_size)).astype(np.float32)
    out = torch.full(prev.shape, -5.0, device="cuda")
    run_weights(plan, four, dev_bf16(batch.q), pool, dev(lse), out, prev=dev(prev), decay=decay, window=window)
    assert plan.device_error() == 0
    want, tol = ref.key_weights(batch, vals, lse, prev, decay, window)
    got, here = out.double().cpu().numpy(), ~np.isnan(want)
    assert np.all(got[~here] == -5.0)                                     # no slot but the plan's tokens'
    assert np.all(np.abs(got[here] - want[here]) <= tol[here] + 1e-37)


LONG = [  # G, D, P, qo, kv, causal, window: every ring of the long form wraps (ten or five Q stages, four accumulators)
    (8, 64, 16, [600, 129, 333], [600, 400, 334], True, 0),
    (16, 128, 32, [700, 130], [700, 131], True, 0),
    (8, 128, 64, [1100], [1190], True, 0),
    (8, 64, 64, [1100], [1190], False, 0),
    (16, 128, 128, [600], [600], False, 0),
    (8, 64, 16, [1200], [1200], True, 700),                               # a window of many steps
    (16, 128, 16, [900], [950], True, 600),
    (1, 64, 16, [1900], [1901], True, 0),
    (20, 64, 64, [650], [700], True, 0),                                  # heads that leave a step's last columns empty
    (20, 128, 16, [1050], [1050], True, 0),
    (12, 64, 16, [1050], [1060], True, 0),
    (12, 128, 128, [700], [700], False, 0),
    (5, 128, 32, [1650], [1650], True, 0),
    (3, 64, 16, [800], [1000], False, 300),
    (130, 64, 16, [70], [300], True, 0),                                  # a row in slices of heads
    (130, 128, 64, [68], [200], False, 40),
    (96, 128, 16, [90], [140], True, 0),
    (43, 64, 32, [150], [200], True, 0),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("G,D,P,qo,kv,causal,window", LONG)
def test_long_form(four, G, D, P, qo, kv, causal, window):
    batch = batch_of(qo, kv, G, 1, D, P, seed=G + D + len(qo), causal=causal)
    check(batch, four, window, 152, ["long"])


SHORT = [
    (8, 64, 16, [1, 5, 70, 130, 33, 2], [17, 5, 200, 130, 64, 1500], True, 0),
    (3, 128, 64, [70, 130, 33], [200, 130, 64], True, 0),
    (16, 64, 128, [70, 130], [200, 400], False, 32),
    (1, 128, 16, [130, 300], [130, 700], True, 0),
    (20, 64, 32, [70, 33], [200, 64], True, 0),
    (12, 128, 32, [70, 130, 33], [200, 130, 640], False, 1),
    (128, 64, 32, [20, 7], [300, 130], True, 0),
    (130, 64, 16, [6, 9], [600, 137], True, 0),
    (130, 128, 16, [5], [900], True, 2),
]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("G,D,P,qo,kv,causal,window", SHORT)
def test_short_form(four, G, D, P, qo, kv, causal, window):
    batch = batch_of(qo, kv, G, 2, D, P, seed=G + D + len(qo), causal=causal)
    check(batch, four, window, 1, ["short"], decay=0.0 if window == 1 else 0.75)


MIXED = [  # D, Hkv, causal, window, SMs of the plan, forms
    (64, 1, True, 0, 8, ["long", "short"]),
    (128, 2, False, 0, 30, ["long", "short"]),
    (64, 2, True, 10, 20, ["long", "short"]),                             # the window leaves both few steps, the prompt few CTAs
    (64, 1, True, 10, 6, ["short", "short"]),                             # apart in the plan, one launch by the window
    (64, 1, True, 0, 1, ["short"]),                                       # the others outlast the prompt
    (64, 1, True, 0, 152, ["long"]),
]


def mixed(D, Hkv, causal):
    more = 6 if D == 128 else 0                       # (the short form of 128 dims asks for more CTAs)
    qo, kv = [3, 2, 1100, 4, 1, 5] + [6] * more, [200, 700, 1150, 129, 300, 1800] + [1500] * more
    return batch_of(qo, kv, 8, Hkv, D, 16, seed=D, causal=causal)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D,Hkv,causal,window,num_sms,want", MIXED)
def test_prompts_beside_few_rows(four, D, Hkv, causal, window, num_sms, want):
    """A long prompt among requests of a few rows on longer contexts: each kind in
    its form where the prompt would outlast the others, else one launch."""
    batch = mixed(D, Hkv, causal)
    check(batch, four, window, num_sms, want)


@pytest.mark.parametrize("four", [False, True])
def test_many_runs_of_tiles(four):
    """Requests whose tiles are one run each, beside prompts whose tiles are all
    runs of their own: more runs than one look at the table covers."""
    rng = np.random.default_rng(2)
    qo = [2, 300] + [int(n) for n in rng.integers(2, 140, 40)]
    kv = [4000, 300] + [int(n + p) for n, p in zip(qo[2:], rng.integers(0, 400, 40))]
    batch = batch_of(qo, kv, 1, 1, 64, 16, seed=4)
    check(batch, four, 0, 152, ["long"])
    check(batch, four, 0, 1, ["short"])


@pytest.mark.parametrize("G,D,num_sms,want", [(20, 64, 152, ["long"]), (20, 128, 152, ["long"]), (12, 64, 152, ["long"]),
                                              (8, 128, 152, ["long"]), (20, 64, 1, ["long"])])
def test_infinite_keys_of_long_prompts(G, D, num_sms, want):
    """A key at minus infinity receives nothing, whatever columns a step leaves
    empty; the others are as without it."""
    n = 65 * (128 // G) + 30
    batch = batch_of([n], [n + 50], G, 1, D, 16, seed=G)
    assert forms(batch, 0, num_sms) == want
    _, pool, vals = pools(batch, False, 4)
    lse = some_lse(batch, vals)
    q = syn.bf16_to_float(batch.q).copy()
    q[..., 0] = np.abs(q[..., 0]) + 1
    q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    plan = make_plan(batch, dev(batch.page_table), num_sms=num_sms)
    zeros = lambda: torch.zeros(batch.num_pages, 1, 16, device="cuda")
    without = plan.key_weights(q, pool, dev(lse), zeros(), decay=0.0).cpu().numpy()
    pool = pool.clone()
    for t in (3, 130, n):
        page, row = int(batch.page_table[t // 16]), t % 16
        pool[page, 0, :, row, 0] = -float("inf")
        without[page, :, row] = 0
    got = plan.key_weights(q, pool, dev(lse), zeros(), decay=0.0).cpu().numpy()
    np.testing.assert_array_equal(got, without)
