"""Page management on the GPU: tables, counts and pools equal to the plain form's,
whatever the calls did before (bit for bit: everything here is copied or counted)."""
import numpy as np
import pytest
import torch

import pages_reference as ref

pytestmark = pytest.mark.gpu


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def dev(x):
    return torch.from_numpy(np.array(x, dtype=np.int32, copy=True).reshape(-1)).cuda()


def pair(rng, num_pages, page_size, refs=None, page_words=(8,), rng_pools=True):
    """The same pools and counts on the device and in the plain form."""
    host = [rng.integers(-2 ** 31, 2 ** 31, (num_pages, w), dtype=np.int64).astype(np.int32) for w in page_words]
    mine = binding().PagePool([torch.from_numpy(h.copy()).cuda() for h in host], page_size,
                              refs=None if refs is None else dev(refs))
    return mine, ref.Pages(host, page_size, refs)


def same(mine, plain, err=None):
    assert mine.refs.tolist() == plain.refs
    for a, b in zip(mine.pools, plain.pools):
        assert np.array_equal(a.cpu().numpy(), b)
    assert mine.device_error() == (plain.err if err is None else err)
    plain.err = 0
    assert mine.device_error() == 0


SIZES = [1, 3, 4, 127, 128, 129, 1000, 32768, 70001]


@pytest.mark.parametrize("num_pages", SIZES)
def test_alloc_and_free(num_pages):
    rng = np.random.default_rng(num_pages)
    refs = (rng.random(num_pages) < 0.6) * rng.integers(1, 4, num_pages)
    mine, plain = pair(rng, num_pages, 16, refs, (4,))
    room = int((refs == 0).sum())
    for n in (0, 1, room // 3, room, 5):                       # the last ones ask for more than there is
        assert mine.alloc(n).tolist() == plain.alloc(n)
        same(mine, plain)
    held = np.repeat(np.arange(num_pages), plain.refs)
    ids = rng.permutation(held)[:len(held) * 2 // 3]
    mine.free(dev(ids))
    plain.free(ids.tolist())
    same(mine, plain)
    assert mine.alloc(num_pages).tolist() == plain.alloc(num_pages)
    same(mine, plain)


def test_free_refuses_what_nothing_holds():
    rng = np.random.default_rng(1)
    mine, plain = pair(rng, 300, 16, [2, 0, 1] * 100)
    ids = [0, 0, 0, 0, 3, 1, 1, 2, 5, 5]
    mine.free(dev(ids))
    plain.free(ids)
    assert plain.err == ref.PAGES
    same(mine, plain)
    ids = [-1, 300, 2 ** 31 - 1, -(2 ** 31), 8, 8] + [9] * 5000
    mine.free(dev(ids))
    plain.free(ids)
    assert plain.err == ref.PAGES | ref.PAGE_ID
    same(mine, plain)


@pytest.mark.parametrize("page_words", [(4,), (8, 4096, 4), (4092, 4100), (40000,), (4,) * 67 + (8,) * 70])
def test_copy(page_words):
    rng = np.random.default_rng(len(page_words))
    mine, plain = pair(rng, 60, 16, None, page_words)
    ids = rng.permutation(60)
    src, dst = np.concatenate([ids[:20], ids[:3]]), ids[20:43]  # one page into several
    mine.copy(dev(src), dev(dst))
    plain.copy(src, dst)
    same(mine, plain)
    src[[0, 5]], dst[[3, 5]] = [60, -1], [-7, 70]
    mine.copy(dev(src), dev(dst))
    plain.copy(src, dst)
    assert plain.err == ref.PAGE_ID
    same(mine, plain)
    none = dev([])
    mine.copy(none, none)
    same(mine, plain)


def test_a_pool_past_4_gb():
    """Offsets beyond 32 bits."""
    pool = torch.zeros(5, 1 << 28, dtype=torch.float32, device="cuda")
    pool[4, -7:], pool[1, 5] = 3.0, 2.0
    mine = binding().PagePool([pool], 16, refs=dev([0, 1, 0, 0, 2]))
    table = dev([4, 1, 4])
    assert mine.compact(table).tolist() == [-1, 1, -1, -1, 0]
    assert table.tolist() == [0, 1, 0] and mine.refs.tolist() == [2, 1, 0, 0, 0] and mine.device_error() == 0
    assert bool((pool[0, -7:] == 3.0).all()) and float(pool[0].sum()) == 21.0 and float(pool[1].sum()) == 2.0


def fork_both(mine, plain, table, indptr, lens, parents, extra=0):
    need = sum(-(-int(lens[b]) // plain.page_size) for b in parents if 0 <= b < len(lens))
    out = torch.full((need + extra,), -77, dtype=torch.int32, device="cuda")
    got, got_indptr = mine.fork(dev(table), dev(indptr), dev(lens), dev(parents), need + extra, out=out)
    want, want_indptr = plain.fork([int(x) for x in table], [int(x) for x in indptr], [int(x) for x in lens], list(parents),
                                   need + extra)
    assert got_indptr.tolist() == want_indptr
    assert got.tolist() == want + [-77] * (need + extra - len(want))
    return want, want_indptr


@pytest.mark.parametrize("num_pages,used,batch,children,page_size", [
    (1, 0, 1, 3, 16), (2, 1, 1, 1, 16), (50, 20, 6, 13, 16), (1000, 700, 40, 200, 64), (33000, 20000, 300, 9000, 128),
    (40000, 30000, 2, 5, 16), (900, 300, 20, 50, 7)])
def test_fork(num_pages, used, batch, children, page_size):
    rng = np.random.default_rng(num_pages + children)
    table, indptr, lens, refs = ref.random_state(rng, num_pages, used, batch, page_size)
    mine, plain = pair(rng, num_pages, page_size, refs, (4, 12))
    parents = [int(b) for b in rng.integers(0, batch, children)]
    out, out_indptr = fork_both(mine, plain, table, indptr, lens, parents, extra=3)
    same(mine, plain)
    # The children are requests as any other: fork them, give the first ones up, compact the rest.
    lens2 = [int(lens[b]) for b in parents]
    second, _ = fork_both(mine, plain, out, out_indptr, lens2, [0, children - 1, 0])
    same(mine, plain)
    mine.free(dev(out))
    plain.free(out)
    same(mine, plain)
    both = np.concatenate([table, second]).astype(np.int32)
    mine_table = dev(both)
    remap = mine.compact(mine_table)
    want, want_remap = plain.compact([int(x) for x in both])
    assert mine_table.tolist() == want and remap.tolist() == want_remap
    same(mine, plain)


def test_fork_and_compact_in_more_pools_than_a_launch_holds():
    rng = np.random.default_rng(20)
    table, indptr, lens, refs = ref.random_state(rng, 60, 30, 6, 16)
    mine, plain = pair(rng, 60, 16, refs, (4, 12, 8, 4100) * 34)
    out, _ = fork_both(mine, plain, table, indptr, lens, [0, 1, 2, 3, 4, 5, 5, 5])
    same(mine, plain)
    mine.free(dev(table))
    plain.free(table.tolist())
    got = dev(out)
    remap = mine.compact(got)
    want, want_remap = plain.compact(out)
    assert got.tolist() == want and remap.tolist() == want_remap
    same(mine, plain)


def test_fork_takes_a_prefix_and_ignores_spare_pages():
    rng = np.random.default_rng(3)
    table, refs = np.array([7, 3, 9, 1]), np.zeros(12, int)
    refs[table] = 1
    mine, plain = pair(rng, 12, 16, refs)
    out, _ = fork_both(mine, plain, table, [0, 4], [20], [0, 0])     # 2 of the 4 pages
    assert out == [7, 0, 7, 2]
    same(mine, plain)


def test_fork_refusals():
    rng = np.random.default_rng(4)
    refs = [1, 1, 1, 1, 0, 0, 1, 1]
    mine, plain = pair(rng, 8, 16, refs)
    table, indptr = [0, 1, 2, 3, 6, 7], [0, 2, 4, 6]
    fork_both(mine, plain, table, indptr, [20, 33, 32], [1, -1, 3, 2 ** 31 - 1, 0, 2])   # 33 tokens on two pages
    assert plain.err == ref.PLAN
    same(mine, plain)
    fork_both(mine, plain, table, indptr, [20, 32, -5], [0, 2, 0])                       # one free page for two children
    assert plain.err == ref.PLAN | ref.PAGES
    same(mine, plain)
    # More entries than fit: refused as a whole.
    out = torch.full((5,), -77, dtype=torch.int32, device="cuda")
    plain.free([4, 5])
    mine.free(dev([4, 5]))
    got, got_indptr = mine.fork(dev(table), dev(indptr), dev([20, 17, 32]), dev([0, 1, 2]), 5, out=out)
    assert got.tolist() == [-77] * 5 and got_indptr.tolist() == [0] * 4
    same(mine, plain, ref.PLAN)
    # Page ids outside the pool: shared entries, and the page to be copied.
    fork_both(mine, plain, [0, 1, 99, 3, 6, -4], indptr, [20, 32, 30], [1, 2])
    assert plain.err & ref.PAGE_ID
    same(mine, plain)
    fork_both(mine, plain, table, [0, 2, 4, 8], [20, 17, 60], [2])                       # past the table's end
    assert plain.err == ref.PLAN
    same(mine, plain)
    got, got_indptr = mine.fork(dev(table), dev(indptr), dev([1, 1, 1]), dev([]), 0)
    assert got_indptr.tolist() == [0] and got.numel() == 0
    same(mine, plain)


@pytest.mark.parametrize("num_pages", SIZES + [1 << 20])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact(num_pages, share):
    rng = np.random.default_rng(num_pages)
    refs = (rng.random(num_pages) < share) * rng.integers(1, 5, num_pages)
    mine, plain = pair(rng, num_pages, 16, refs, (4,) if num_pages > 5000 else (4, 4100))
    table = np.repeat(np.arange(num_pages), refs)
    table = rng.permutation(table)[:20000]
    got = dev(table)
    remap = mine.compact(got)
    want, want_remap = plain.compact(table.tolist())
    assert got.tolist() == want and remap.tolist() == want_remap
    same(mine, plain)
    again = mine.compact(got)                                        # nothing left to move
    assert got.tolist() == want
    assert again.tolist() == [p if n else -1 for p, n in enumerate(plain.refs)]
    same(mine, plain)


def test_compact_flags_bad_entries():
    rng = np.random.default_rng(9)
    mine, plain = pair(rng, 10, 16, [0, 1, 0, 0, 1, 0, 0, 2, 0, 0])
    table = [7, -1, 10, 4, 0, 1, 9]
    got = dev(table)
    mine.compact(got)
    want, _ = plain.compact(table)
    assert got.tolist() == want == [0, -1, 10, 2, -1, 1, -1]
    assert plain.err == ref.PAGE_ID | ref.PAGES
    same(mine, plain)
    mine.compact(dev([]))


def test_a_captured_step_replays():
    """Free, fork, alloc and copy in one graph, replayed over counts that go on changing."""
    rng = np.random.default_rng(11)
    table, indptr, lens, refs = ref.random_state(rng, 500, 260, 9, 16)
    refs[table[:2]] += 5                                         # given up below, never to the last
    mine, plain = pair(rng, 500, 16, refs, (4, 64))
    parents = [0, 4, 4, 8, 2]
    need = sum(-(-int(lens[b]) // 16) for b in parents)
    t, i, l, p = dev(table), dev(indptr), dev(lens), dev(parents)
    out, out_indptr, ids = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (need, 6, 7))
    src = t[:7].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mine.fork(t, i, l, p, need, out=out, indptr_out=out_indptr)
        mine.alloc(7, out=ids)
        mine.copy(src, ids)
        mine.free(src[:2])
    plain.refs = mine.refs.tolist()
    for step in range(3):
        if step == 1:                                            # other requests forked, other lengths
            lens[0], parents[0] = max(1, lens[0]) // 2, 0
            l.copy_(dev(lens))
        if step == 2:
            mine.refs[table[0]] += 2
            plain.refs[table[0]] += 2
        graph.replay()
        torch.cuda.synchronize()
        want, want_indptr = plain.fork(table.tolist(), indptr.tolist(), lens.tolist(), parents, need)
        new = plain.alloc(7)
        plain.copy(table[:7].tolist(), new)
        plain.free(table[:2].tolist())
        assert out_indptr.tolist() == want_indptr and out.tolist()[:len(want)] == want and ids.tolist() == new
        same(mine, plain)


def test_calls_on_another_stream():
    rng = np.random.default_rng(12)
    table, indptr, lens, refs = ref.random_state(rng, 2000, 900, 9, 32)
    mine, plain = pair(rng, 2000, 32, refs, (256,))
    side = torch.cuda.Stream()
    args = [dev(x) for x in (table, indptr, lens, [1, 5, 8])]
    need = sum(-(-int(lens[b]) // 32) for b in (1, 5, 8))
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(1000000)                                    # the current stream is late
    out, _ = mine.fork(*args, need, stream=side)
    mine.free(args[0][:20], stream=side)
    ids = mine.alloc(30, stream=side)
    remap = mine.compact(out, stream=side)
    side.synchronize()
    want, _ = plain.fork(table.tolist(), indptr.tolist(), lens.tolist(), [1, 5, 8], need)
    plain.free(table[:20].tolist())
    new = plain.alloc(30)
    want, want_remap = plain.compact(want)
    assert ids.tolist() == new and out.tolist() == want and remap.tolist() == want_remap
    same(mine, plain)


def test_the_binding_refuses():
    B = binding()
    pool = torch.zeros(8, 4, device="cuda")
    for bad in (dict(pools=[]), dict(pools=[pool.cpu()]), dict(pools=[pool, pool[:7]]), dict(pools=[pool[:, :3].contiguous()]),
                dict(pools=[pool.t()]), dict(page_size=0), dict(refs=torch.zeros(8, device="cuda")),
                dict(refs=torch.zeros(9, dtype=torch.int32, device="cuda")), dict(pools=[torch.zeros(0, 4, device="cuda")]),
                dict(refs=torch.zeros(9, dtype=torch.int32, device="cuda")[1:])):
        with pytest.raises((TypeError, ValueError)):
            B.PagePool(**{**dict(pools=[pool], page_size=16), **bad})
    pages = B.PagePool([pool], 16)
    ids = dev([1, 2])
    for call in (lambda: pages.free(ids.long()), lambda: pages.free(ids[None]), lambda: pages.copy(ids, ids[:1]),
                 lambda: pages.alloc(2, out=ids[:1]), lambda: pages.compact(ids.cpu()), lambda: pages.fork(ids, ids, ids, ids, 2),
                 lambda: pages.fork(ids, dev([0, 1, 2]), ids, ids, 2, out=ids[:1])):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_counts_past_31_bits_are_refused():
    """None is cut to the 32 bits that the C entry points take."""
    B = binding()
    pages = B.PagePool([torch.zeros(8, 4, device="cuda")], 16)
    for n in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError):
            pages.alloc(n)
    ids, many = dev([1, 2]), torch.empty(1 << 31, dtype=torch.int32, device="cuda")
    for call in (lambda: pages.free(many), lambda: pages.fork(ids, dev([0, 1, 2]), ids, many, 2)):
        with pytest.raises(ValueError):
            call()
    assert not pages.refs.any() and pages.device_error() == 0
