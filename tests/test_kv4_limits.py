"""CPU checks of the sizes that the compressed cache's entry points take: what
their 32-bit index arithmetic would not hold is refused before a launch (no
pages are listed, so nothing would be launched either way)."""
import ctypes

import pytest

from test_abi import INVALID, OK, UNSUPPORTED, lib   # noqa: F401  (lib: the built library's fixture)

P = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("Hkv,page,D,want", [(64, 1 << 20, 128, UNSUPPORTED), (1 << 17, 1024, 64, UNSUPPORTED),
                                             (4, 1 << 30, 64, UNSUPPORTED), ((1 << 31) - 1, (1 << 31) - 16, 128, UNSUPPORTED),
                                             (63, 1 << 20, 128, OK), ((1 << 17) - 1, 1024, 64, OK), (8, 4096, 64, OK)])
def test_expand_refuses_pages_beyond_32_bit_indices(lib, Hkv, page, D, want):   # noqa: F811
    """A page's K (or V) half has Hkv * page_size * D / 8 items of eight dims; the
    kernel steps through them in int32 and adds a step below that count to an
    index below it: under 2^30 both fit."""
    assert (Hkv * page * D // 8 >= 1 << 30) == (want == UNSUPPORTED)
    assert lib.attn_expand_kv4(P, 4, Hkv, page, D, P, 0, 1.0, 1.0, P, None, None) == want


ODD2 = ctypes.c_void_p(0x10002)


def test_expand_refuses_a_misaligned_error_word(lib):   # noqa: F811
    assert lib.attn_expand_kv4(P, 4, 2, 16, 64, P, 1, 1.0, 1.0, P, ODD2, None) == INVALID
