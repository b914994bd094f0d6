"""Key weights and eviction on the GPU against plain fp64 forms
(kv4_reference), and the compressed cache's operators run together.

Key weights: fp32 throughout; the reference returns the bound on such an
evaluation's error beside the values.  Eviction copies: compared exactly.
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from helpers import make_plan, syn
from test_kv4_gpu import batch_of, binding, check_decode, dev, dev_bf16

pytestmark = pytest.mark.gpu


def pools(batch, four, seed=0):
    """(host pool, device pool, fp64 values) in either form, unused slots poisoned."""
    D, P, Hkv = batch.head_dim, batch.page_size, batch.num_kv_heads
    rng = np.random.default_rng(seed)
    if four:
        pool = ref.random_pool(rng, batch.num_pages, Hkv, P, D)
        ref.poison_unused(pool, batch)
        return pool, dev(pool), ref.values(pool, D)
    full = syn.make_batch("x", batch.qo_lens, batch.kv_lens, batch.num_qo_heads, Hkv, D, P,
                          pool_pages=batch.num_pages, seed=seed + 77)
    batch.page_table = full.page_table          # the poison follows this table
    return full.kv_pool, dev_bf16(full.kv_pool), syn.bf16_to_float(full.kv_pool).astype(np.float64)


def some_lse(batch, vals):
    """Log-sum-exps near the true ones (any value would do)."""
    lse = np.log(np.repeat(batch.kv_lens, batch.qo_lens).astype(np.float64))[:, None]
    return (lse + np.random.default_rng(1).normal(0.5, 0.5, size=(batch.total_rows, batch.num_qo_heads))).astype(np.float32)


def run_weights(plan, four, q, pool, lse, weights, **kw):
    return (plan.key_weights_kv4 if four else plan.key_weights)(q, pool, lse, weights, **kw)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("G,D,P,causal", [(8, 64, 16, True), (3, 128, 64, True), (16, 64, 128, False), (1, 128, 16, True),
                                          (20, 64, 32, True), (12, 128, 32, False)])
def test_key_weights_match_reference(four, G, D, P, causal):
    qo = [1, 1, 1, 0, 5, 70, 130, 1, 33]
    kv = [1, 17, 300, 20, 5, 200, 130, 129, 64]
    batch = batch_of(qo, kv, G, 2, D, P, seed=G + P, causal=causal)
    _, pool, vals = pools(batch, four, seed=G)
    plan = make_plan(batch, dev(batch.page_table))
    lse = some_lse(batch, vals)
    rng = np.random.default_rng(3)
    prev = rng.exponential(size=(batch.num_pages, 2, P)).astype(np.float32)
    for decay, window in ((1.0, 0), (0.75, 32), (0.0, 1)):
        before = np.full_like(prev, np.nan) if decay == 0 else prev
        out = torch.full(prev.shape, -5.0, device="cuda")
        run_weights(plan, four, dev_bf16(batch.q), pool, dev(lse), out, prev=dev(before), decay=decay, window=window)
        assert plan.device_error() == 0
        want, tol = ref.key_weights(batch, vals, lse, before, decay, window)
        got = out.double().cpu().numpy()
        here = ~np.isnan(want)
        assert np.all(got[~here] == -5.0)                                 # no slot but the plan's tokens'
        assert np.all(np.abs(got[here] - want[here]) <= tol[here] + 1e-37), (decay, window)


@pytest.mark.parametrize("four,D,G,P", [(False, 64, 8, 16), (True, 128, 5, 64), (False, 128, 16, 32)])
def test_key_weights_of_longer_prompts(four, D, G, P):
    """Enough rows and heads that every ring of the kernel wraps several times,
    with a prefix, a window, and rows that end inside a tile."""
    batch = batch_of([600, 129, 333], [600, 400, 334], G, 1, D, P, seed=D + G)
    _, pool, vals = pools(batch, four, seed=3)
    plan = make_plan(batch, dev(batch.page_table))
    lse = some_lse(batch, vals)
    prev = np.random.default_rng(5).exponential(size=(batch.num_pages, 1, P)).astype(np.float32)
    for window in (0, 200):
        out = torch.full(prev.shape, -5.0, device="cuda")
        run_weights(plan, four, dev_bf16(batch.q), pool, dev(lse), out, prev=dev(prev), window=window)
        assert plan.device_error() == 0
        want, tol = ref.key_weights(batch, vals, lse, prev, 1.0, window)
        got, here = out.double().cpu().numpy(), ~np.isnan(want)
        assert np.all(got[~here] == -5.0)
        assert np.all(np.abs(got[here] - want[here]) <= tol[here] + 1e-37), window


def test_key_weights_mask_foreign_rows_and_keys():
    """Query rows of a neighbour that are NaN, NaN keys past the end, and a NaN
    key among the request's own, which spoils its own weight alone."""
    batch = batch_of([40, 70], [40, 75], 4, 2, 64, 16, seed=9)
    _, pool, vals = pools(batch, False, 4)
    lse, q = some_lse(batch, vals), batch.q.copy()
    q[:40] = 0x7FC0                                              # request 0's rows
    own = batch.page_table[batch.kv_indptr[1]]                   # request 1's tokens 0..15
    pool = pool.clone()
    pool[own, 0, 1, 3] = float("nan")
    vals = pool.double().cpu().numpy()
    plan = make_plan(batch, dev(batch.page_table))
    w = plan.key_weights(dev_bf16(q), pool, dev(lse), torch.zeros(batch.num_pages, 2, 16, device="cuda"), decay=0.0)
    batch.q = batch.q.copy()
    want, tol = ref.key_weights(batch, np.where(np.isnan(vals), 0, vals), lse, np.zeros(w.shape), 0.0, 0)
    pages = batch.page_table[batch.kv_indptr[1]:batch.kv_indptr[2]]
    got = w.double().cpu().numpy()
    assert np.isnan(got[own, 1, 3])
    got[own, 1, 3] = want[own, 1, 3]
    here = ~np.isnan(want[pages])
    assert np.all(np.abs(got[pages] - want[pages])[here] <= tol[pages][here] + 1e-37)


def test_key_weights_in_place_and_again():
    """weights is its own prev: two steps add up, the new token starts at zero,
    and equal calls give equal bits."""
    batch = batch_of([1, 1, 40], [700, 33, 90], 8, 2, 64, 16, seed=4)
    _, pool, vals = pools(batch, False, 2)
    plan = make_plan(batch, dev(batch.page_table))
    lse, q = some_lse(batch, vals), dev_bf16(batch.q)
    w = torch.full((batch.num_pages, 2, 16), 7.0, device="cuda")
    first = plan.key_weights(q, pool, dev(lse), w.clone(), decay=0.0)
    plan.key_weights(q, pool, dev(lse), w)                                # decay 1 on 7.0
    want, tol = ref.key_weights(batch, vals, lse, np.full(w.shape, 7.0), 1.0, 0)
    here = ~np.isnan(want)
    assert np.all(np.abs(w.double().cpu().numpy()[here] - want[here]) <= tol[here] + 8 * 2.0 ** -24)
    second = plan.key_weights(q, pool, dev(lse), torch.empty_like(w), decay=0.0)
    assert torch.equal(first[dev(here)].view(torch.int32), second[dev(here)].view(torch.int32))


def test_key_weights_sum_to_the_attention_on_keys():
    """With the lse that decode returned and no sink, a row's weights add up to
    the number of query heads."""
    batch = batch_of([1] * 3, [1, 250, 3000], 8, 2, 64, 16, seed=8, with_sinks=False)
    pool, d_pool, _ = pools(batch, True, 5)
    plan = make_plan(batch, dev(batch.page_table))
    lse = torch.empty(3, 16, device="cuda")
    plan.decode_kv4(dev_bf16(batch.q), d_pool, lse=lse)
    w = plan.key_weights_kv4(dev_bf16(batch.q), d_pool, lse, torch.zeros(batch.num_pages, 2, 16, device="cuda"), decay=0.0)
    for b in range(3):
        pages = torch.from_numpy(batch.page_table[batch.kv_indptr[b]:batch.kv_indptr[b + 1]]).long().cuda()
        total = w[pages].double().sum((0, 2)).cpu().numpy()
        # lse itself is within 2^-12 (its own test); a head's share is exp of that.
        assert np.all(np.abs(total - 8) <= 8 * 2.0 ** -11)


# ------------------------------------------------------------------- eviction

def evict_reference(batch, pool, weights, budget, recent, out_pages, pool_out, weights_out, four):
    """In place on the host copies; returns kept."""
    D, P, Hkv = batch.head_dim, batch.page_size, batch.num_kv_heads
    kept = np.full((batch.batch_size, Hkv, budget), -1, dtype=np.int32)
    src, w_src = pool.copy(), weights.copy()

    def row(x, page, half, g, t):
        if not four:
            return x[page, half, g, t % P],
        blk, t = x[page, half, g, (t % P) // 16], t % 16
        return blk[t * (D // 2):(t + 1) * (D // 2)], blk[8 * D + t * (D // 16):8 * D + (t + 1) * (D // 16)]

    for b in range(batch.batch_size):
        n = int(batch.kv_lens[b])
        pages = batch.page_table[batch.kv_indptr[b]:batch.kv_indptr[b + 1]]
        for g in range(Hkv):
            w = np.array([w_src[pages[t // P], g, t % P] for t in range(n)])
            keep = ref.evict(w, n, budget, recent)
            kept[b, g, :len(keep)] = keep
            for j, t in enumerate(keep):
                to = out_pages[b][j // P]
                weights_out[to, g, j % P] = w[t]
                for half in (0, 1):
                    for a, c in zip(row(pool_out, to, half, g, j), row(src, pages[t // P], half, g, t)):
                        a[:] = c
    return kept


def weights_like(rng, shape):
    """Heavy tails, many zeros, equal values, and a few NaN, infinities and -0."""
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    w[rng.random(shape) < 0.3] = 0
    w[rng.random(shape) < 0.05] = -0.0
    w[rng.random(shape) < 0.3] = 0.5
    w[rng.random(shape) < 0.01] = np.nan
    w[rng.random(shape) < 0.01] = np.inf
    w[rng.random(shape) < 0.01] = -np.inf
    w[rng.random(shape) < 0.01] = -1.5
    return w


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,P,Hkv,budget,recent", [(64, 16, 2, 100, 16), (128, 64, 1, 33, 33), (64, 128, 3, 700, 1),
                                                   (128, 32, 2, 1, 0), (64, 16, 1, 5000, 10), (128, 16, 2, 129, 0)])
def test_evict_matches_reference(four, in_place, D, P, Hkv, budget, recent):
    kv = [1, 16, 99, 100, 101, 0, 650, 1200]
    batch = batch_of([0] * len(kv), kv, 2, Hkv, D, P, seed=budget)
    pool, d_pool, _ = pools(batch, four, 1)
    weights = weights_like(np.random.default_rng(budget), (batch.num_pages, Hkv, P))
    plan = make_plan(batch, dev(batch.page_table))
    lens = plan.evicted_lens(budget)
    np.testing.assert_array_equal(lens, np.minimum(kv, budget))
    need = -(-lens // P)
    call = plan.evict_kv4 if four else plan.evict_kv
    d_w = dev(weights)
    if in_place:
        out_pages = [batch.page_table[batch.kv_indptr[b]:] for b in range(len(kv))]
        want_pool, want_w = pool.copy(), weights.copy()
        kept = call(d_w, d_pool, budget, recent)
        got_pool, got_w = d_pool, d_w
    else:
        n_out = int(need.sum()) + 2
        table = np.random.default_rng(7).permutation(n_out)[:need.sum()].astype(np.int32)
        out_pages = np.split(table, np.cumsum(need)[:-1])
        want_pool = np.full((n_out,) + pool.shape[1:], 99, dtype=pool.dtype)
        want_w = np.full((n_out, Hkv, P), 5.0, dtype=np.float32)
        got_pool = dev(want_pool) if four else dev_bf16(want_pool)
        got_w = dev(want_w)
        kept = call(d_w, d_pool, budget, recent, page_table_out=dev(table), kv_out=got_pool, weights_out=got_w)
    want_kept = evict_reference(batch, pool, weights, budget, recent, out_pages, want_pool, want_w, four)
    assert plan.device_error() == 0
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    got = got_pool.cpu().numpy() if four else got_pool.view(torch.int16).cpu().numpy().view(np.uint16)
    np.testing.assert_array_equal(got, want_pool)
    np.testing.assert_array_equal(got_w.cpu().numpy().view(np.uint32), want_w.view(np.uint32))


def test_evict_into_other_pages_of_the_same_pool():
    batch = batch_of([0, 0], [90, 300], 2, 2, 64, 16, seed=2, pool_pages=60)
    pool, d_pool, _ = pools(batch, False, 3)
    weights = weights_like(np.random.default_rng(1), (60, 2, 16))
    plan = make_plan(batch, dev(batch.page_table))
    free = np.setdiff1d(np.arange(60), batch.page_table).astype(np.int32)[:6]     # 3 pages each for 48 tokens
    want_pool, want_w = pool.copy(), weights.copy()
    want = evict_reference(batch, pool, weights, 48, 8, [free[:3], free[3:]], want_pool, want_w, False)
    d_w = dev(weights)
    kept = plan.evict_kv(d_w, d_pool, 48, 8, page_table_out=dev(free))
    np.testing.assert_array_equal(kept.cpu().numpy(), want)
    np.testing.assert_array_equal(d_pool.view(torch.int16).cpu().numpy().view(np.uint16), want_pool)
    np.testing.assert_array_equal(d_w.cpu().numpy().view(np.uint32), want_w.view(np.uint32))


def test_evict_long_rows_and_equal_weights():
    """One long request; all weights equal (the oldest are kept), then two values."""
    n, budget = 20000, 6001
    batch = batch_of([1], [n], 1, 1, 64, 128, seed=1)
    plan = make_plan(batch, dev(batch.page_table))
    pool = torch.zeros(batch.num_pages, 2, 1, 128, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.full((batch.num_pages, 1, 128), 0.25, device="cuda")
    kept = plan.evict_kv(w, pool, budget, 1).cpu().numpy()[0, 0]
    np.testing.assert_array_equal(kept, np.r_[np.arange(budget - 1), n - 1])
    flat = np.full(n, 1.0, dtype=np.float32)
    flat[::7] = np.nextafter(np.float32(1), np.float32(2))            # differ in the last bit of the key
    host = np.zeros((batch.num_pages, 1, 128), dtype=np.float32)
    t = np.arange(n)
    host[batch.page_table[t // 128], 0, t % 128] = flat
    kept = plan.evict_kv(dev(host), pool, budget, 0).cpu().numpy()[0, 0]
    np.testing.assert_array_equal(kept, ref.evict(flat, n, budget, 0))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv,Hkv,budget,recent", [([50001, 40], 1, 20011, 100), ([12003] + [17] * 89, 2, 5000, 7)])
def test_evict_rows_longer_than_shared_memory(in_place, kv, Hkv, budget, recent):
    """Rows whose weights are read in chunks, for few rows (a CTA takes a whole
    SM) and for many."""
    P, D = 64, 64
    batch = batch_of([0] * len(kv), kv, 1, Hkv, D, P, seed=len(kv))
    weights = weights_like(np.random.default_rng(3), (batch.num_pages, Hkv, P))
    plan = make_plan(batch, dev(batch.page_table))
    pool = torch.arange(batch.num_pages * 2 * Hkv * P, device="cuda", dtype=torch.int32)   # every row its number
    pool = pool.view(-1, 1).expand(-1, D // 2).contiguous().view(torch.bfloat16).view(batch.num_pages, 2, Hkv, P, D)
    before, d_w = pool.clone(), dev(weights)
    if in_place:
        kept, out, w_out = plan.evict_kv(d_w, pool, budget, recent), pool, d_w
        tables = [batch.page_table[batch.kv_indptr[b]:] for b in range(len(kv))]
    else:
        need = -(-plan.evicted_lens(budget) // P)
        table = np.random.default_rng(7).permutation(int(need.sum())).astype(np.int32)
        tables = np.split(table, np.cumsum(need)[:-1])
        out = torch.zeros(len(table), 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
        w_out = torch.zeros(len(table), Hkv, P, device="cuda")
        kept = plan.evict_kv(d_w, pool, budget, recent, page_table_out=dev(table), kv_out=out, weights_out=w_out)
    assert plan.device_error() == 0
    kept, out, before = kept.cpu().numpy(), out.view(torch.int32).cpu().numpy(), before.view(torch.int32).cpu().numpy()
    w_out = w_out.cpu().numpy()
    for b in range(len(kv)):
        pages = batch.page_table[batch.kv_indptr[b]:batch.kv_indptr[b + 1]]
        for g in range(Hkv):
            w = weights[pages, g].reshape(-1)[:kv[b]]
            want = ref.evict(w, kv[b], budget, recent)
            np.testing.assert_array_equal(kept[b, g, :len(want)], want)
            assert np.all(kept[b, g, len(want):] == -1)
            j = np.arange(len(want))
            to = np.asarray(tables[b])[j // P]
            np.testing.assert_array_equal(w_out[to, g, j % P].view(np.uint32), w[want].view(np.uint32))
            for half in (0, 1):
                np.testing.assert_array_equal(out[to, half, g, j % P], before[pages[want // P], half, g, want % P])


def test_evict_bad_pages():
    """Bad ids are recorded and skipped; other requests are served."""
    batch = batch_of([0, 0], [64, 64], 2, 1, 64, 16, seed=2)
    pool, d_pool, _ = pools(batch, False, 3)
    weights = weights_like(np.random.default_rng(1), (batch.num_pages, 1, 16))
    pt = dev(batch.page_table)
    plan = make_plan(batch, pt)
    pt[1] = batch.num_pages
    out = torch.full((4, 2, 1, 16, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    w_out = torch.full((4, 1, 16), 9.0, device="cuda")
    kept = plan.evict_kv(dev(weights), d_pool, 32, 4, page_table_out=dev(np.array([0, 1, 2, -1], dtype=np.int32)),
                         kv_out=out, weights_out=w_out)
    assert plan.device_error() == 1
    pages = batch.page_table[4:8]
    want = ref.evict(weights[pages, 0].reshape(-1), 64, 32, 4)
    np.testing.assert_array_equal(kept.cpu().numpy()[1, 0], want)
    np.testing.assert_array_equal(w_out[2, 0].cpu().numpy().view(np.uint32), weights[pages, 0].reshape(-1)[want[:16]].view(np.uint32))
    assert torch.all(out[3] == 9.0)


def test_refusals():
    b = binding()
    batch = batch_of([1, 1], [20, 30], 4, 2, 64, 16)
    _, pool, _ = pools(batch, False)
    plan = make_plan(batch, dev(batch.page_table))
    q, lse = dev_bf16(batch.q), torch.zeros(2, 8, device="cuda")
    w = torch.zeros(batch.num_pages, 2, 16, device="cuda")
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(b.AttnError):
            plan.key_weights(q, pool, lse, w, decay=bad)
    with pytest.raises(b.AttnError):
        plan.key_weights(q, pool, lse, w, window=-1)
    with pytest.raises(ValueError):
        plan.key_weights(q, pool, lse, w[:-1])
    with pytest.raises(TypeError):
        plan.key_weights(q, pool, lse.double(), w)
    with pytest.raises(TypeError):
        plan.key_weights_kv4(q, pool, lse, w)
    for budget, recent in ((0, 0), (4, 5), (4, -1)):
        with pytest.raises(ValueError):
            plan.evict_kv(w, pool, budget, recent)
    with pytest.raises(ValueError):
        plan.evict_kv(w, pool, 8, 0, weights_out=w.clone())               # no pages to go to
    with pytest.raises(ValueError):
        plan.evict_kv(w, pool, 8, 0, page_table_out=torch.zeros(3, dtype=torch.int32, device="cuda"))   # two are needed
    with pytest.raises(ValueError):
        plan.evict_kv(w, pool, 8, 0, page_table_out=torch.zeros(2, dtype=torch.int32, device="cuda"),
                      kv_out=pool.clone(), weights_out=w[:2].contiguous())
    assert not torch.any(w)


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("four", [False, True])
def test_serving_loop(four):
    """A few decode steps with key weights, then an eviction in place and a step
    over the shrunk cache: outputs against attention over exactly the kept keys."""
    b, (Hkv, G, D, P), budget = binding(), (2, 4, 64, 16), 40
    kv = np.array([90, 33, 41])
    rng = np.random.default_rng(11)
    total = int((-(-(kv + 8) // P)).sum())
    table = rng.permutation(total + 4)[:total].astype(np.int32)
    page_of = np.concatenate([[0], np.cumsum(-(-(kv + 8) // P))])
    d_table = dev(table)
    n_pool = total + 4
    if four:
        host = ref.random_pool(rng, n_pool, Hkv, P, D)
        cache = dev(host)
    else:
        cache = dev_bf16(syn.bf16_bits(rng.standard_normal((n_pool, 2, Hkv, P, D), dtype=np.float32)))
    weights = torch.zeros(n_pool, Hkv, P, device="cuda")
    prev_w = np.zeros((n_pool, Hkv, P))

    def host_values():
        return ref.values(cache.cpu().numpy(), D) if four else cache.double().cpu().numpy()

    def step(lens, seed, first):
        """One decode step of requests that now hold `lens` tokens."""
        batch = syn.make_batch("s", [1] * 3, lens, Hkv * G, Hkv, D, P, seed=seed, fill_pool=False)
        need = -(-np.asarray(lens) // P)
        own = np.concatenate([table[page_of[i]:page_of[i] + need[i]] for i in range(3)]).astype(np.int32)
        batch.page_table, batch.pool_pages = own, n_pool
        plan = make_plan(batch, dev(own))
        k_new, v_new = syn.new_kv_rows(batch, seed)
        lse = torch.empty(3, Hkv * G, device="cuda")
        if four:
            plan.append_kv4(dev_bf16(k_new), dev_bf16(v_new), cache)
            out, _ = plan.decode_kv4(dev_bf16(batch.q), cache, dev(batch.sinks), lse=lse)
            plan.key_weights_kv4(dev_bf16(batch.q), cache, lse, weights, decay=0.0 if first else 1.0)
        else:
            plan.append_kv(dev_bf16(k_new), dev_bf16(v_new), cache)
            out, _ = plan.decode(dev_bf16(batch.q), cache, dev(batch.sinks), lse=lse)
            plan.key_weights(dev_bf16(batch.q), cache, lse, weights, decay=0.0 if first else 1.0)
        assert plan.device_error() == 0
        vals = host_values()
        want, want_lse, mag = ref.attention(batch, vals)
        err = np.abs(out.double().cpu().numpy() - want)
        # P in bf16 (half a step: 2^-8, in the sum and in what normalises it) or in f16: the coarser bound serves both.
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag)
        w, tol = ref.key_weights(batch, vals, lse.cpu().numpy(), prev_w, 0.0 if first else 1.0, 0)
        got = weights.double().cpu().numpy()
        here = ~np.isnan(w)
        assert np.all(np.abs(got - w)[here] <= tol[here] + 1e-37)
        prev_w[:] = got
        return plan, batch

    for s in range(3):
        plan, batch = step(kv + 1 + s, 100 + s, s == 0)
    before, w_before = host_values(), weights.cpu().numpy()
    kept = (plan.evict_kv4 if four else plan.evict_kv)(weights, cache, budget, 8).cpu().numpy()
    lens = plan.evicted_lens(budget)
    after = host_values()
    for i in range(3):
        n = int(batch.kv_lens[i])
        pages = batch.page_table[batch.kv_indptr[i]:batch.kv_indptr[i + 1]]
        for g in range(Hkv):
            w = w_before[pages, g].reshape(-1)[:n]
            want = ref.evict(w, n, budget, 8)
            np.testing.assert_array_equal(kept[i, g, :len(want)], want)
            for half in (0, 1):
                old = before[pages, half, g].reshape(-1, D)[want]
                new = after[pages, half, g].reshape(-1, D)[:len(want)]
                np.testing.assert_array_equal(new, old)
    prev_w[:] = weights.double().cpu().numpy()
    step(lens + 1, 200, False)                                          # goes on over the shrunk cache


def test_captured_step_replays_on_new_inputs():
    """Append, decode, key weights and an eviction into spare pages in one CUDA
    graph, replayed on new rows; equal to the same calls made eagerly."""
    batch = batch_of([1, 1, 1], [130, 7, 512], 8, 2, 64, 16, seed=21)
    pool, d_pool, _ = pools(batch, True, 9)
    plan = make_plan(batch, dev(batch.page_table))
    q = dev_bf16(batch.q)
    k_new, v_new = (dev_bf16(x) for x in syn.new_kv_rows(batch, 1))
    sinks, budget = dev(batch.sinks), 64
    need = int((-(-plan.evicted_lens(budget) // 16)).sum())
    table = torch.arange(need, dtype=torch.int32, device="cuda")
    prev = torch.rand(batch.num_pages, 2, 16, device="cuda")
    bufs = dict(out=torch.empty_like(q), lse=torch.empty(3, 16, device="cuda"), weights=torch.zeros_like(prev),
                kept=torch.empty(3, 2, budget, dtype=torch.int32, device="cuda"),
                kv_out=torch.zeros(need, *d_pool.shape[1:], dtype=torch.uint8, device="cuda"),
                weights_out=torch.zeros(need, 2, 16, device="cuda"),
                back=torch.empty(need, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda"))

    def calls():
        plan.append_kv4(k_new, v_new, d_pool)
        plan.decode_kv4(q, d_pool, sinks, bufs["out"], bufs["lse"])
        plan.key_weights_kv4(q, d_pool, bufs["lse"], bufs["weights"], prev=prev)
        plan.evict_kv4(bufs["weights"], d_pool, budget, 8, kept=bufs["kept"], page_table_out=table, kv_out=bufs["kv_out"],
                       weights_out=bufs["weights_out"])
        binding().attn_expand_kv4(bufs["kv_out"], table, 64, buf=bufs["back"])

    calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            calls()
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k_new, v_new):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen).to(torch.bfloat16))
        prev.copy_(torch.rand(prev.shape, device="cuda", generator=gen))
        for t in bufs.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = {k: t.clone() for k, t in bufs.items()}
        calls()
        torch.cuda.synchronize()
        for k, t in bufs.items():
            assert torch.equal(t.view(torch.uint8), replayed[k].view(torch.uint8)), k
    assert plan.device_error() == 0


def test_another_stream():
    """All operators on a stream given explicitly, with outputs they allocate."""
    batch = batch_of([1, 1], [300, 50], 4, 2, 64, 16, seed=31)
    pool, d_pool, _ = pools(batch, True, 9)
    plan = make_plan(batch, dev(batch.page_table))
    q, sinks = dev_bf16(batch.q), dev(batch.sinks)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lse = torch.empty(2, 8, device="cuda")
    w = torch.zeros(batch.num_pages, 2, 16, device="cuda")
    torch.cuda.synchronize()
    out, _ = plan.decode_kv4(q, d_pool, sinks, lse=lse, stream=s)
    plan.key_weights_kv4(q, d_pool, lse, w, decay=0.0, stream=s)
    kept = plan.evict_kv4(w, d_pool, 20, 4, stream=s)
    s.synchronize()
    check_decode(batch, pool, out, lse)
    assert int(kept[0, 0, -1]) == 299 and int(kept[1, 1, -1]) == 49


def test_captured_branches():
    """Kernels of two branches of one graph, with copies and fills between them,
    each after what it reads: equal to the same calls one after the other."""
    batch = batch_of([1, 1, 1], [700, 33, 1500], 8, 2, 64, 16, seed=33)
    pool, d_pool, _ = pools(batch, True, 9)
    plan = make_plan(batch, dev(batch.page_table))
    q, q_next = dev_bf16(batch.q), torch.empty_like(dev_bf16(batch.q))
    k_new, v_new = (dev_bf16(x) for x in syn.new_kv_rows(batch, 1))
    sinks, budget = dev(batch.sinks), 40
    pages = dev(batch.page_table)
    bufs = dict(out=torch.empty_like(q), lse=torch.empty(3, 16, device="cuda"),
                weights=torch.zeros(batch.num_pages, 2, 16, device="cuda"),
                kept=torch.empty(3, 2, budget, dtype=torch.int32, device="cuda"),
                back=torch.empty(len(pages), 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda"))

    def calls(side):
        main = torch.cuda.current_stream()
        bufs["weights"].zero_()
        plan.append_kv4(k_new, v_new, d_pool)
        if side is not None:
            side.wait_stream(main)
        with torch.cuda.stream(side if side is not None else main):
            q_next.copy_(q)
            binding().attn_expand_kv4(d_pool, pages, 64, buf=bufs["back"])
            q_next.mul_(0.5)
        plan.decode_kv4(q, d_pool, sinks, bufs["out"], bufs["lse"])
        plan.key_weights_kv4(q, d_pool, bufs["lse"], bufs["weights"], prev=bufs["weights"], decay=0.5)
        if side is not None:
            main.wait_stream(side)
        plan.decode_kv4(q_next, d_pool, sinks, bufs["out"], bufs["lse"])
        plan.key_weights_kv4(q_next, d_pool, bufs["lse"], bufs["weights"], prev=bufs["weights"], decay=0.5)
        plan.evict_kv4(bufs["weights"], d_pool, budget, 8, kept=bufs["kept"])

    first_pool = d_pool.clone()
    calls(None)
    torch.cuda.synchronize()
    want, want_pool = {k: t.clone() for k, t in bufs.items()}, d_pool.clone()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            calls(side)
    for _ in range(3):
        d_pool.copy_(first_pool)
        for t in bufs.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d_pool, want_pool)
        for k, t in bufs.items():
            assert torch.equal(t.view(torch.uint8), want[k].view(torch.uint8)), k
    assert plan.device_error() == 0


@pytest.mark.parametrize("n,budget,recent", [(700, 1, 0), (700, 130, 3), (700, 350, 0), (700, 520, 64), (700, 699, 0),
                                             (20000, 9000, 100), (20000, 17000, 1)])
def test_evict_orders_all_values(n, budget, recent):
    """Weights of either sign and size, zeros of either sign, infinities and
    NaNs, each many times; and no others but one value."""
    rng = np.random.default_rng(n + budget)
    some = np.array([-np.inf, -3e38, -1.0, -1e-38, -1e-45, -0.0, 0.0, 1e-45, 1e-38, 1.0, np.nextafter(np.float32(1), 2),
                     3e38, np.inf, np.nan], dtype=np.float32)
    Hkv, P = len(some) + 3, 16
    pages = -(-n // P)
    flat = np.full((Hkv, pages * P), np.nan, dtype=np.float32)
    flat[:3, :n] = rng.choice(some, (3, n))
    flat[3:, :n] = some[:, None]
    batch = batch_of([1], [n], 1, Hkv, 64, P)
    plan = make_plan(batch, dev(batch.page_table))
    host = np.zeros((batch.num_pages, Hkv, P), dtype=np.float32)
    host[batch.page_table] = flat.reshape(Hkv, pages, P).transpose(1, 0, 2)
    pool = torch.zeros(batch.num_pages, 2, Hkv, P, 64, dtype=torch.bfloat16, device="cuda")
    w = dev(host)
    kept = plan.evict_kv(w, pool, budget, recent).cpu().numpy()[0]
    moved = w.cpu().numpy()[batch.page_table].transpose(1, 0, 2).reshape(Hkv, -1)
    for g in range(Hkv):
        want = ref.evict(flat[g], n, budget, recent)
        np.testing.assert_array_equal(kept[g], want, err_msg=str(g))
        np.testing.assert_array_equal(moved[g, :budget].view(np.uint32), flat[g, want].view(np.uint32), err_msg=str(g))


def test_after_another_streams_event():
    """A call behind an event of another stream, and behind a call of the same
    kind, waits for both: its rows, its weights and its plan's lists arrive late."""
    first, second = (batch_of([1, 1], kv, 8, 2, 64, 16, seed=41) for kv in ([900, 60], [60, 900]))
    pool, d_pool, _ = pools(first, True, 9)
    table = dev(first.page_table)
    q = dev_bf16(second.q)
    want_plan = make_plan(second, table)
    want, want_lse = want_plan.decode_kv4(q, d_pool, lse=torch.empty(2, 16, device="cuda"))
    want_w = want_plan.key_weights_kv4(q, d_pool, want_lse, torch.zeros(first.num_pages, 2, 16, device="cuda"), decay=0.0)
    want_kept = want_plan.evict_kv4(want_w.clone(), d_pool.clone(), 20, 4)
    plan = make_plan(first, table)
    torch.cuda.synchronize()
    side, late = torch.cuda.Stream(), torch.zeros_like(q)
    for _ in range(3):
        late.zero_()
        weights, lse = torch.zeros_like(want_w), torch.empty_like(want_lse)
        torch.cuda.synchronize()
        plan.decode_kv4(late, d_pool, lse=torch.empty_like(lse))
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)
            late.copy_(q)
            next_plan = binding().Plan(second.qo_indptr, second.kv_indptr, table, second.last_page_len, 16, 2, 64, 16,
                                       causal=second.causal, sm_scale=second.sm_scale, num_pages=second.num_pages)
            torch.cuda._sleep(2_000_000)
        torch.cuda.current_stream().wait_stream(side)
        out, _ = next_plan.decode_kv4(late, d_pool, lse=lse)
        next_plan.key_weights_kv4(late, d_pool, lse, weights, decay=0.0)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            kept = next_plan.evict_kv4(weights.clone(), d_pool.clone(), 20, 4)
        torch.cuda.synchronize()
        for got, expect in ((out, want), (lse, want_lse), (weights, want_w), (kept, want_kept)):
            assert torch.equal(got.view(torch.uint8), expect.view(torch.uint8))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D,P,budget,recent", [(64, 16, 48, 5), (128, 16, 33, 0), (128, 64, 90, 90), (64, 32, 1, 1)])
def test_evict_many_rows(four, D, P, budget, recent):
    """More rows than SMs, out of place, with pages outside the pools among them."""
    rng = np.random.default_rng(budget)
    kv = [0, 1, 1200] + [int(n) for n in rng.integers(0, 150, 87)]
    batch = batch_of([0] * len(kv), kv, 1, 2, D, P, seed=budget)
    pool, d_pool, _ = pools(batch, four, 1)
    weights = weights_like(rng, (batch.num_pages, 2, P))
    plan = make_plan(batch, dev(batch.page_table))
    need = -(-plan.evicted_lens(budget) // P)
    n_out = int(need.sum()) + 2
    table = rng.permutation(n_out)[:need.sum()].astype(np.int32)
    out_pages = np.split(table, np.cumsum(need)[:-1])
    want_pool = np.full((n_out,) + pool.shape[1:], 99, dtype=pool.dtype)
    want_w = np.full((n_out, 2, P), 5.0, dtype=np.float32)
    call, pool0, w0 = plan.evict_kv4 if four else plan.evict_kv, want_pool.copy(), want_w.copy()
    out = lambda: (dev(pool0) if four else dev_bf16(pool0), dev(w0))
    host = lambda t: t.cpu().numpy() if four else t.view(torch.int16).cpu().numpy().view(np.uint16)
    got_pool, got_w = out()
    kept = call(dev(weights), d_pool, budget, recent, page_table_out=dev(table), kv_out=got_pool, weights_out=got_w)
    want_kept = evict_reference(batch, pool, weights, budget, recent, out_pages, want_pool, want_w, four)
    assert plan.device_error() == 0
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    np.testing.assert_array_equal(host(got_pool), want_pool)
    np.testing.assert_array_equal(got_w.cpu().numpy().view(np.uint32), want_w.view(np.uint32))
    # Request 2's first receiving page lies outside: it alone stays as it was.
    first = int(need[:2].sum())
    bad = table.copy()
    bad[first] = n_out
    got_pool, got_w = out()
    kept = call(dev(weights), d_pool, budget, recent, page_table_out=dev(bad), kv_out=got_pool, weights_out=got_w)
    assert plan.device_error() == 1
    want_pool[table[first]], want_w[table[first]] = pool0[table[first]], w0[table[first]]
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    np.testing.assert_array_equal(host(got_pool), want_pool)
    np.testing.assert_array_equal(got_w.cpu().numpy().view(np.uint32), want_w.view(np.uint32))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("G,D,P,n,causal", [(32, 64, 16, 400, True), (20, 128, 64, 410, True), (128, 64, 32, 75, False),
                                            (130, 64, 16, 60, True), (130, 128, 16, 9, True)])
def test_key_weights_of_many_heads(four, G, D, P, n, causal):
    """Few rows of many heads to a step, more than a step's columns among them;
    long and short lists of steps."""
    batch = batch_of([n, 3], [n + 37, 130], G, 1, D, P, seed=G + n, causal=causal)
    _, pool, vals = pools(batch, four, seed=3)
    plan = make_plan(batch, dev(batch.page_table))
    lse = some_lse(batch, vals)
    prev = np.random.default_rng(5).exponential(size=(batch.num_pages, 1, P)).astype(np.float32)
    for window in (0, 50):
        out = torch.full(prev.shape, -5.0, device="cuda")
        run_weights(plan, four, dev_bf16(batch.q), pool, dev(lse), out, prev=dev(prev), window=window)
        assert plan.device_error() == 0
        want, tol = ref.key_weights(batch, vals, lse, prev, 1.0, window)
        got, here = out.double().cpu().numpy(), ~np.isnan(want)
        assert np.all(got[~here] == -5.0)
        assert np.all(np.abs(got[here] - want[here]) <= tol[here] + 1e-37), window


@pytest.mark.parametrize("G", [1, 3, 8, 12, 20])
def test_key_weights_of_infinite_keys(G):
    """A key at minus infinity receives nothing, whatever heads a tile leaves
    empty; the others are as without it."""
    batch = batch_of([1, 40, 1], [50, 70, 40], G, 2, 64, 16, seed=G)
    _, pool, vals = pools(batch, False, 4)
    lse = some_lse(batch, vals)
    q = syn.bf16_to_float(batch.q).copy()
    q[..., 0] = np.abs(q[..., 0]) + 1
    q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    plan = make_plan(batch, dev(batch.page_table))
    zeros = lambda: torch.zeros(batch.num_pages, 2, 16, device="cuda")
    without = plan.key_weights(q, pool, dev(lse), zeros(), decay=0.0).cpu().numpy()
    pool = pool.clone()
    at = [(batch.page_table[batch.kv_indptr[b] + t // 16], t % 16)
          for b, t in ((0, 3), (1, 20), (2, 33))]
    for page, row in at:
        pool[int(page), 0, :, row, 0] = -float("inf")
        without[int(page), :, row] = 0
    got = plan.key_weights(q, pool, dev(lse), zeros(), decay=0.0).cpu().numpy()
    np.testing.assert_array_equal(got, without)
