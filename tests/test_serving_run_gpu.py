"""The operators around attention as a serving loop uses them together: prompts are
turned and appended, attended, forked into beams, stepped (new pages where a page
is full) with cross attention to shared encoder states, thinned out, compacted and
stepped again.  Every attention output is compared with a plain 64-bit form over
each request's own list of keys and values, which knows nothing of pages.

Tolerance: that of test_cross_gpu.py, whose roundings are the same.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def plain(q, k, v, scale, causal_from=None):
    """q [rows, Hq, D] over k, v [T, Hkv, D]; row i sees keys 0 .. causal_from + i.  Returns out and sum w |v|."""
    G = q.shape[1] // k.shape[1]
    k, v = (x.double().repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("rhd,thd->rht", q.double(), k) * scale
    if causal_from is not None:
        t = torch.arange(k.shape[0], device=q.device)
        s = s.masked_fill(t[None, None] > causal_from + torch.arange(len(q), device=q.device)[:, None, None], -float("inf"))
    w = torch.softmax(s, -1)
    return torch.einsum("rht,thd->rhd", w, v), torch.einsum("rht,thd->rhd", w, v.abs())


def close(out, want, mag):
    err = (out.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -13 + 2.0 ** -11) * mag + 1e-30
    assert bool((err <= tol).all()), float((err / tol).max())


class Loop:
    """A batch of requests on one layer: page tables on the device, lengths on the host, and what they should hold."""

    def __init__(self, Hq, Hkv, D, P, num_pages, enc_lens, seed, sms):
        from paged_kv_attention_sink_gb300 import binding
        self.B, self.Hq, self.Hkv, self.D, self.P = binding, Hq, Hkv, D, P
        self.sms = sms                                     # what cross attention is planned for: 1 takes every kernel
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.full((num_pages, 2, Hkv, P, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pages = binding.PagePool([self.pool], P)
        self.rope = binding.Rope((1000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32), axis=[p % 3 for p in range(D // 2)])
        self.enc_lens, self.enc_start = enc_lens, np.concatenate([[0], np.cumsum(enc_lens)[:-1]]).tolist()
        self.enc = self.rows(sum(enc_lens), 2 * Hkv)
        self.lens, self.kv, self.enc_of = [], [], []       # per request: tokens, [(k, v)] so far, encoder
        self.table = torch.empty(0, dtype=torch.int32, device="cuda")

    def rows(self, n, heads):
        return torch.randn(n, heads, self.D, device="cuda", generator=self.g).to(torch.bfloat16)

    def counts(self):
        return [-(-n // self.P) for n in self.lens]

    def split(self):
        return list(torch.split(self.table, self.counts()))

    def step(self, new):
        """Request b gets new[b] tokens: pages, rotary positions and append, attention, cross attention."""
        tables, want_pages = self.split(), []
        for b, n in enumerate(new):
            self.lens[b] += n
            want_pages.append(-(-self.lens[b] // self.P) - len(tables[b]))
        fresh = torch.split(self.pages.alloc(sum(want_pages)), want_pages)
        self.table = torch.cat([x for pair in zip(tables, fresh) for x in pair])
        qo, indptr = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(self.counts())])
        last = [n - (c - 1) * self.P for n, c in zip(self.lens, self.counts())]
        plan = self.B.Plan(qo, indptr, self.table, last, self.Hq, self.Hkv, self.D, self.P, num_pages=len(self.pool))
        qkv = self.rows(qo[-1], self.Hq + 2 * self.Hkv)
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:-self.Hkv], qkv[:, -self.Hkv:]
        pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(self.lens, new)]).to(torch.int32)
        pos = torch.stack([pos, pos // 7, pos % 7])
        q = plan.append_kv_rope(self.rope, pos, q, k, v, self.pool)
        out = torch.full_like(q, float("nan"))
        plan.prefill(q, self.pool, out=out)
        plan.decode(q, self.pool, out=out)
        turned = self.rope.apply(pos, qkv[:, self.Hq:-self.Hkv])
        for b, m in enumerate(new):
            r = slice(qo[b], qo[b + 1])
            self.kv[b] = [torch.cat((x, y[r])) for x, y in zip(self.kv[b], (turned, v))]
            close(out[r], *plain(q[r], *self.kv[b], self.D ** -0.5, self.lens[b] - m))
        # Requests of one encoder are neighbours: their rows are one sequence's.
        first = [b for b in range(len(new)) if b == 0 or self.enc_of[b] != self.enc_of[b - 1]]
        cross = self.B.CrossPlan([qo[b] for b in first] + [qo[-1]], [self.enc_start[self.enc_of[b]] for b in first],
                                 [self.enc_lens[self.enc_of[b]] for b in first], len(self.enc), self.Hq, self.Hkv, self.D,
                                 num_sms=self.sms)
        got, _ = cross.attend(out, self.enc[:, :self.Hkv], self.enc[:, self.Hkv:])
        for b in range(len(new)):
            e, r = self.enc_of[b], slice(qo[b], qo[b + 1])
            if self.enc_lens[e] == 0:
                assert not got[r].any()
                continue
            states = self.enc[self.enc_start[e]:self.enc_start[e] + self.enc_lens[e]]
            close(got[r], *plain(out[r], states[:, :self.Hkv], states[:, self.Hkv:], self.D ** -0.5))
        assert plan.device_error() == 0 and cross.device_error() == 0 and self.pages.device_error() == 0

    def add(self, n, enc):
        for _ in range(n):
            self.lens.append(0)
            self.kv.append([torch.zeros(0, self.Hkv, self.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
            self.enc_of.append(enc)

    def fork(self, parents):
        """One more request per parent, behind it."""
        n = self.counts()
        i32 = dict(dtype=torch.int32, device="cuda")
        table, indptr = self.pages.fork(self.table, torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32),
                                        torch.tensor(self.lens, **i32), torch.tensor(parents, **i32), sum(n[p] for p in parents))
        assert indptr.tolist() == np.concatenate([[0], np.cumsum([n[p] for p in parents])]).tolist()
        tables = [[t] for t in self.split()]
        children = list(torch.split(table, [n[p] for p in parents]))
        order = sorted(range(len(self.lens) + len(parents)),
                       key=lambda i: (i, 0) if i < len(n) else (parents[i - len(n)], i))
        flat = [t[0] for t in tables] + children
        pick = lambda own, of: [own[i] if i < len(n) else of[parents[i - len(n)]] for i in order]
        self.table = torch.cat([flat[i] for i in order])
        self.kv = [list(x) for x in pick(self.kv, self.kv)]
        self.lens, self.enc_of = pick(self.lens, self.lens), pick(self.enc_of, self.enc_of)

    def drop(self, gone):
        tables = self.split()
        self.pages.free(torch.cat([tables[b] for b in gone]))
        keep = [b for b in range(len(self.lens)) if b not in gone]
        self.table = torch.cat([tables[b] for b in keep])
        self.lens, self.kv, self.enc_of = ([x[b] for b in keep] for x in (self.lens, self.kv, self.enc_of))


@pytest.mark.parametrize("Hq,Hkv,D,P,sms", [(8, 2, 64, 16, 0), (16, 4, 128, 32, 1), (16, 2, 64, 16, 1)])
def test_prompts_beams_and_compaction(Hq, Hkv, D, P, sms):
    loop = Loop(Hq, Hkv, D, P, 90, [70, 1500, 0], seed=D, sms=sms)
    for e in (0, 1, 2):
        loop.add(1, e)
    loop.step([5 * P, 37, 2 * P - 1])           # prompts: a full last page, a ragged one, one to be filled
    loop.fork([0, 0, 1, 1, 1, 2])
    assert (loop.pages.refs == 3).sum() == 5    # the first prompt's pages, all full
    for _ in range(3):                          # past a page's end
        loop.step([1] * 9)
    loop.fork([4, 7])
    loop.step([1, 4, 1, 2, 1, 1, 3, 1, 1, 1, 1])   # some verify drafts
    loop.drop([0, 3, 5, 9])
    held = int((loop.pages.refs > 0).sum())
    remap = loop.pages.compact(loop.table)
    assert int(loop.table.max()) < held and int(remap.max()) == held - 1
    loop.pool[held:] = float("nan")             # nothing is left back there
    for _ in range(2):
        loop.step([1] * 7)
    loop.drop(range(7 - 1))
    loop.pages.free(loop.table)
    assert not loop.pages.refs.any() and loop.pages.device_error() == 0


def test_compressed_pages_and_weights_are_forked_and_compacted_alike():
    """A child's 4-bit pages and key weights are its parent's, wherever they lie: equal queries give equal bits."""
    from paged_kv_attention_sink_gb300 import binding
    Hq, Hkv, D, P, n = 16, 4, 64, 32, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [70, 5 * P, 9]
    counts = [-(-m // P) for m in lens]
    pool = torch.zeros(binding.kv4_cache_shape(n, Hkv, P, D), dtype=torch.uint8, device="cuda")
    weights = torch.zeros(n, Hkv, P, device="cuda")
    pages = binding.PagePool([pool, weights], P)
    pages.alloc(3)                                              # others' pages
    table = pages.alloc(sum(counts))

    def plan_of(table, lens, qo):
        c = [-(-m // P) for m in lens]
        return binding.Plan(np.concatenate([[0], np.cumsum(qo)]), np.concatenate([[0], np.cumsum(c)]), table,
                            [m - (k - 1) * P for m, k in zip(lens, c)], Hq, Hkv, D, P, num_pages=n)

    rows = lambda m, h: torch.randn(m, h, D, device="cuda", generator=g).to(torch.bfloat16)
    plan_of(table, lens, lens).append_kv4(rows(sum(lens), Hkv), rows(sum(lens), Hkv), pool)
    q = rows(3, Hq)
    plan = plan_of(table, lens, [1, 1, 1])
    out, lse = plan.decode_kv4(q, pool, lse=torch.empty(3, Hq, device="cuda"))
    plan.key_weights_kv4(q, pool, lse, weights, decay=0.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    parents = [2, 0, 0, 1]
    child, indptr = pages.fork(table, torch.tensor(np.concatenate([[0], np.cumsum(counts)]), **i32), torch.tensor(lens, **i32),
                               torch.tensor(parents, **i32), sum(counts[b] for b in parents))
    pages.free(table)
    want = weights[table.long()]
    pages.compact(child)
    assert int((pages.refs > 0).sum()) == int(child.max()) + 1
    forked = plan_of(child, [lens[b] for b in parents], [1] * 4)
    got, got_lse = forked.decode_kv4(q[parents], pool, lse=torch.empty(4, Hq, device="cuda"))
    assert torch.equal(got, out[parents]) and torch.equal(got_lse, lse[parents])
    first = np.concatenate([[0], np.cumsum(counts)])
    order = torch.tensor(np.concatenate([np.arange(first[b], first[b + 1]) for b in parents]), device="cuda")
    assert torch.equal(weights[child.long()], want[order])
    assert pages.device_error() == 0 and forked.device_error() == 0
