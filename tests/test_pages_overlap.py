"""Page calls refuse arrays that overlap where one of them is written: the scans read
their inputs twice and would index by what changed in between (CPU: refused before the
device is looked at, at pointers that are never dereferenced)."""
import ctypes
import itertools

import pytest

from test_abi import INVALID, OK, lib   # noqa: F401  (lib: the built library's fixture)

PAGES, BATCH, N, TABLE, OUT = 100, 3, 5, 40, 30


def at(address):
    return ctypes.c_void_p(address)


def pools():
    return (ctypes.c_void_p * 1)(0x90000000), (ctypes.c_int64 * 1)(512), 1


def fork(lib, a, n=N):
    return lib.attn_pages_fork(at(a["refs"]), PAGES, at(a["table"]), TABLE, at(a["indptr"]), at(a["lens"]), BATCH, 16,
                               at(a["parents"]), n, at(a["out"]), at(a["indptr_out"]), OUT, *pools(), at(a["scratch"]), None, None)


def compact(lib, a):
    return lib.attn_pages_compact(at(a["refs"]), PAGES, at(a["table"]), TABLE, at(a["remap"]), *pools(), at(a["scratch"]), None, None)


FORK = dict(refs=PAGES, table=TABLE, indptr=BATCH + 1, lens=BATCH, parents=N, out=OUT, indptr_out=N + 1, scratch=4 + 2 * N)
COMPACT = dict(refs=PAGES, table=TABLE, remap=PAGES, scratch=4 + PAGES)
READ = {"table", "indptr", "lens", "parents"}


def placed(sizes):
    """Each array at an address of its own."""
    return {name: 0x10000 * (i + 1) for i, name in enumerate(sizes)}


@pytest.mark.parametrize("call,sizes,read", [(fork, FORK, READ), (compact, COMPACT, set())])
def test_every_pair_that_is_written(lib, call, sizes, read):
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are accepted would run")
    ok = call(lib, placed(sizes))
    assert ok != INVALID                                   # (no device here: the launch fails)
    for x, y in itertools.permutations(sizes, 2):
        apart = x in read and y in read
        a = placed(sizes)
        for address in (a[x], a[x] + 4 * sizes[x] - 4):    # y begins at x's first word, at its last one
            if y == "refs":
                address &= ~15                             # (refs' own alignment)
            if address + 4 * sizes[y] <= a[x] or address >= a[x] + 4 * sizes[x]:
                continue
            assert (call(lib, {**a, y: address}) == INVALID) == (not apart), (x, y)
        after = (a[x] + 4 * sizes[x] + 15) & ~15
        assert call(lib, {**a, y: after}) == ok            # side by side


def test_a_fork_of_nobody_reads_nothing(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls that are accepted would run")
    a = placed(FORK)
    assert fork(lib, {**a, "indptr": a["indptr_out"], "parents": a["out"]}, n=0) != INVALID


def test_ids_inside_the_counts(lib):
    refs = 0x10000
    for inside in (refs, refs + 4 * PAGES - 4, refs - 4 * (N - 1)):
        assert lib.attn_pages_alloc(at(refs), PAGES, N, at(inside), None, None) == INVALID
        assert lib.attn_pages_free(at(refs), PAGES, at(inside), N, None, None) == INVALID
    assert lib.attn_pages_alloc(at(refs), PAGES, 0, at(refs), None, None) == OK
    assert lib.attn_pages_free(at(refs), PAGES, at(refs), 0, None, None) == OK


@pytest.mark.parametrize("call,sizes", [(fork, FORK), (compact, COMPACT)])
def test_every_array_is_looked_at_for_itself(lib, call, sizes):
    """NULL and misaligned, with everything else sound."""
    for name in sizes:
        for value in (0, 2):
            a = placed(sizes)
            a[name] = a[name] + value if value else 0
            assert call(lib, a) == INVALID, (name, value)
