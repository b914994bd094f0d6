"""Requests that share pages after a fork are evicted into new pages: the ones that go on
with the old pages keep every bit, whoever is evicted first, and the evicted ones equal
a request evicted in place that shares nothing."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [70, 80])            # a last page that is copied; full pages alone
@pytest.mark.parametrize("four", [False, True])
def test_evicted_into_new_pages(D, length, four):
    from paged_kv_attention_sink_gb300 import binding
    Hq, Hkv, P, n, budget, recent = 4, 2, 16, 60, 37, 5
    g = torch.Generator(device="cuda").manual_seed(length)
    pool = torch.zeros(binding.kv4_cache_shape(n, Hkv, P, D) if four else (n, 2, Hkv, P, D),
                       dtype=torch.uint8 if four else torch.bfloat16, device="cuda")
    weights = torch.rand(n, Hkv, P, device="cuda", generator=g)
    pages = binding.PagePool([pool, weights], P)
    pages.alloc(2)                                         # others' pages
    count = -(-length // P)
    table = pages.alloc(count)

    def plan_of(table, lens, qo):
        c = [-(-m // P) for m in lens]
        return binding.Plan(np.concatenate([[0], np.cumsum(qo)]), np.concatenate([[0], np.cumsum(c)]), table,
                            [m - (k - 1) * P for m, k in zip(lens, c)], Hq, Hkv, D, P, num_pages=n)

    rows = lambda m, h: torch.randn(m, h, D, device="cuda", generator=g).to(torch.bfloat16)
    whole = plan_of(table, [length], [length])
    (whole.append_kv4 if four else whole.append_kv)(rows(length, Hkv), rows(length, Hkv), pool)
    q = rows(1, Hq)
    decode = lambda plan, q, pool: (plan.decode_kv4 if four else plan.decode)(q, pool, lse=torch.empty(len(q), Hq, device="cuda"))
    evict = lambda plan, *a, **kw: (plan.evict_kv4 if four else plan.evict_kv)(*a, **kw)

    alone, alone_weights = pool.clone(), weights.clone()   # the same request where nobody shares
    alone_kept = evict(plan_of(table, [length], [1]), alone_weights, alone, budget, recent)
    want = decode(plan_of(table[:-(-budget // P)].contiguous(), [budget], [1]), q, alone)

    i32 = dict(dtype=torch.int32, device="cuda")
    child, _ = pages.fork(table, torch.tensor([0, count], **i32), torch.tensor([length], **i32), torch.tensor([0, 0], **i32),
                          2 * count)
    before, before_weights = pool[table.long()].clone(), weights[table.long()].clone()
    out = decode(plan_of(table, [length], [1]), q, pool)

    fresh = pages.alloc(2 * -(-budget // P))
    children = plan_of(child, [length, length], [1, 1])
    kept = evict(children, weights, pool, budget, recent, page_table_out=fresh)
    pages.free(child)
    assert torch.equal(kept, alone_kept.expand(2, -1, -1))
    assert torch.equal(pool[table.long()], before) and torch.equal(weights[table.long()], before_weights)
    assert all(torch.equal(x, y) for x, y in zip(decode(plan_of(table, [length], [1]), q, pool), out))
    both = decode(plan_of(fresh, [budget, budget], [1, 1]), q.expand(2, -1, -1).contiguous(), pool)
    for x, y in zip(both, want):
        assert torch.equal(x, y.expand(2, *y.shape[1:]))

    # The parent's pages are its own again: in place from here on.
    assert pages.refs[table.long()].tolist() == [1] * count
    evict(plan_of(table, [length], [1]), weights, pool, budget, recent)
    for x, y in zip(decode(plan_of(table[:-(-budget // P)].contiguous(), [budget], [1]), q, pool), want):
        assert torch.equal(x, y)
    assert pages.device_error() == 0 and children.device_error() == 0
