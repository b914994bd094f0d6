"""CPU checks of the page management's entry points: arguments are refused with
a status before anything reaches the device (the pointers here are never
dereferenced there), and the plain form is checked for what it promises."""
import ctypes

import numpy as np
import pytest

import pages_reference as ref
from test_abi import INVALID, OK, lib   # noqa: F401  (lib: the built library's fixture)

P, ODD2, ODD4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10004)


def pools(ptrs=(0x20000,), sizes=(512,)):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(sizes))(*sizes), len(ptrs)


def alloc(lib, refs=P, num_pages=9, n=0, ids=P, err=P):
    return lib.attn_pages_alloc(refs, num_pages, n, ids, err, None)


def free(lib, refs=P, num_pages=9, ids=P, n=0, err=P):
    return lib.attn_pages_free(refs, num_pages, ids, n, err, None)


def copy(lib, pl=pools(), num_pages=9, src=P, dst=P, n=0, err=P):
    return lib.attn_pages_copy(*pl, num_pages, src, dst, n, err, None)


A, B = ctypes.c_void_p(0x30000), ctypes.c_void_p(0x40000)


def fork(lib, refs=P, num_pages=9, table=P, table_len=2, indptr=P, lens=P, batch=2, size=16, parents=P, n=1, out=A, out_indptr=B,
         out_len=1, pl=pools(), scratch=P, err=P):
    return lib.attn_pages_fork(refs, num_pages, table, table_len, indptr, lens, batch, size, parents, n, out, out_indptr, out_len, *pl,
                               scratch, err, None)


def compact(lib, refs=P, num_pages=9, table=P, n=1, remap=P, pl=pools(), scratch=P, err=P):
    return lib.attn_pages_compact(refs, num_pages, table, n, remap, *pl, scratch, err, None)


def test_nothing_to_do(lib):
    assert alloc(lib) == OK and alloc(lib, ids=None, err=None) == OK
    assert free(lib) == OK and free(lib, ids=None, err=None) == OK
    assert copy(lib) == OK and copy(lib, src=None, dst=None) == OK and copy(lib, pl=(None, None, 0)) == OK


@pytest.mark.parametrize("bad", [dict(refs=None), dict(refs=ODD4), dict(num_pages=0), dict(num_pages=-1), dict(err=ODD2)])
def test_bad_state(lib, bad):
    for call in (alloc, free, fork, compact):
        assert call(lib, **bad) == INVALID


@pytest.mark.parametrize("call,bad", [
    (alloc, dict(n=-1)), (alloc, dict(n=1, ids=None)), (alloc, dict(n=1, ids=ODD2)), (free, dict(n=-1)), (free, dict(n=1 << 31)),
    (free, dict(n=1, ids=None)), (free, dict(n=1, ids=ODD2)), (copy, dict(n=-1)), (copy, dict(n=1 << 31)), (copy, dict(num_pages=0)),
    (copy, dict(n=1, src=None)), (copy, dict(n=1, dst=ODD2)), (copy, dict(err=ODD2)), (fork, dict(batch=-1)), (fork, dict(size=0)),
    (fork, dict(n=-1)), (fork, dict(out_len=-1)), (fork, dict(out_len=1 << 31)), (fork, dict(table=None)), (fork, dict(table_len=-1)), (fork, dict(table_len=1 << 31)), (fork, dict(indptr=ODD2)),
    (fork, dict(lens=None)), (fork, dict(parents=None)), (fork, dict(out=None)), (fork, dict(out_indptr=None)),
    (fork, dict(out=P)), (fork, dict(out=ctypes.c_void_p(0x10004))), (fork, dict(out=ctypes.c_void_p(0xfffc), out_len=2)),
    (fork, dict(out_indptr=P)), (fork, dict(out_indptr=ctypes.c_void_p(0x10008))), (fork, dict(scratch=None)), (fork, dict(scratch=ODD2)), (compact, dict(n=-1)), (compact, dict(n=1 << 31)),
    (compact, dict(table=None)), (compact, dict(table=ODD2)), (compact, dict(remap=None)), (compact, dict(scratch=None))])
def test_bad_arguments(lib, call, bad):
    assert call(lib, **bad) == INVALID


@pytest.mark.parametrize("pl", [(None, None, 1), (None, None, -1), pools((0,)), pools((0x20008,)), pools(sizes=(0,)),
                                pools(sizes=(24,)), pools(sizes=(-16,)), pools((0x20000, 0x20001), (16, 16))])
def test_bad_pools(lib, pl):
    for call in (copy, fork, compact):
        assert call(lib, pl=pl) == INVALID


def test_scratch_size(lib):
    assert [lib.attn_pages_scratch(n) for n in (-3, 0, 1, 1 << 31)] == [4, 4, 6, 4 + (1 << 32)]


def test_plain_compaction_keeps_every_request():
    rng = np.random.default_rng(0)
    for n, used in ((1, 0), (1, 1), (40, 17), (40, 39), (64, 64)):
        table, indptr, lens, refs = ref.random_state(rng, n, used, 5, 16)
        data = rng.integers(0, 1000, (n, 3))
        before = data[table].copy()
        pages = ref.Pages([data], 16, refs)
        out, remap = pages.compact(table.tolist())
        assert pages.err == 0 and sorted(out) == list(range(used)) and np.array_equal(data[np.array(out, int)], before)
        assert [r > 0 for r in pages.refs] == [p < used for p in range(n)]


def test_plain_fork_shares_and_copies():
    data = np.arange(8)
    pages = ref.Pages([data], 4, [1, 1, 1, 0, 0, 1, 0, 0])
    out, indptr = pages.fork([5, 0, 1, 2], [0, 2, 4], [6, 8], [0, 1, 0], 6)
    assert (out, indptr) == ([5, 3, 1, 2, 5, 4], [0, 2, 4, 6])
    assert pages.refs == [1, 2, 2, 1, 1, 3, 0, 0] and data.tolist() == [0, 1, 2, 0, 0, 5, 6, 7] and pages.err == 0
