"""CPU checks of the compressed cache's C entry points: arguments are refused
with a status before anything reaches the device (the pointers here are never
dereferenced), and the plain quantiser that the GPU tests use is itself checked
by brute force."""
import ctypes

import numpy as np
import pytest

import kv4_reference as ref
from test_abi import INVALID, OK, UNSUPPORTED, lib, plan   # noqa: F401  (lib: the built library's fixture)

NOT_BOUND = 5
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def calls(lib, h, scale=1.0, decay=1.0, window=0, budget=4, recent=1):
    return {
        "append": lib.attn_append_kv4(h, P, P, scale, scale, P, None),
        "decode": lib.attn_decode_kv4(h, P, P, scale, scale, None, P, None, None),
        "weights": lib.attn_key_weights(h, P, P, P, P, decay, window, P, None),
        "weights4": lib.attn_key_weights_kv4(h, P, P, scale, P, P, decay, window, P, None),
        "evict": lib.attn_evict_kv(h, P, P, budget, recent, P, P, 10, P, P, None),
        "evict4": lib.attn_evict_kv4(h, P, P, budget, recent, P, P, 10, P, P, None),
    }


def test_unbound_null_ragged_and_graph_plans_are_refused(lib):
    st, h, _ = plan(lib, [1], [2], [4])
    assert st == OK
    assert set(calls(lib, h).values()) == {NOT_BOUND}
    lib.attn_plan_destroy(h)
    assert set(calls(lib, None).values()) == {INVALID}
    g, r, ws = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.attn_graph_plan(8, 16, 2, 64, 16, ctypes.c_float(0.125), 1024, 8 * 4096, P, 152, ctypes.byref(g),
                               ctypes.byref(ws)) == OK
    ind = np.array([0, 4], dtype=np.int32)
    assert lib.attn_plan_ragged(ind.ctypes.data, ind.ctypes.data, 1, 16, 2, 64, 1, 0.125, 152, ctypes.byref(r),
                                ctypes.byref(ws)) == OK
    for h in (g, r):
        assert set(calls(lib, h).values()) == {INVALID}
        lib.attn_plan_destroy(h)


def test_kv_lens(lib):
    st, h, _ = plan(lib, [1, 0, 5, 0], [3, 0, 1, 7], [4, 0, 16, 1])
    lens = np.full(5, -9, dtype=np.int32)
    assert lib.attn_plan_get_kv_lens(h, lens.ctypes.data, 4) == OK
    assert lens.tolist() == [36, 0, 16, 97, -9]
    assert lib.attn_plan_get_kv_lens(h, lens.ctypes.data, -1) == INVALID
    assert lib.attn_plan_get_kv_lens(h, None, 2) == INVALID
    assert lib.attn_plan_get_kv_lens(None, lens.ctypes.data, 2) == INVALID
    lib.attn_plan_destroy(h)


@pytest.mark.parametrize("bad", [0.0, -1.0, 1.5, float("nan"), float("inf"), 2.0 ** 41, 2.0 ** -41])
def test_pool_scales_are_powers_of_two(lib, bad):
    st, h, _ = plan(lib, [1], [2], [4])
    assert lib.attn_decode_kv4(h, P, P, bad, 1.0, None, P, None, None) == INVALID
    assert lib.attn_decode_kv4(h, P, P, 1.0, bad, None, P, None, None) == INVALID
    assert lib.attn_expand_kv4(P, 4, 2, 16, 64, P, 1, bad, 1.0, P, None, None) == INVALID
    assert lib.attn_expand_kv4(P, 4, 2, 16, 64, P, 1, 1.0, bad, P, None, None) == INVALID
    lib.attn_plan_destroy(h)


def test_expand_argument_checks(lib):
    assert lib.attn_expand_kv4(P, 4, 2, 16, 64, None, 0, 1.0, 1.0, None, None, None) == OK      # nothing to do
    assert lib.attn_expand_kv4(P, 4, 2, 16, 96, P, 1, 1.0, 1.0, P, None, None) == UNSUPPORTED
    assert lib.attn_expand_kv4(P, 4, 2, 24, 64, P, 1, 1.0, 1.0, P, None, None) == UNSUPPORTED
    for args in ((P, 0, 2, 16, 64, P, 1), (P, 4, 0, 16, 64, P, 1), (P, 4, 2, 16, 64, P, -1), (None, 4, 2, 16, 64, P, 1),
                 (P, 4, 2, 16, 64, None, 1), (ODD, 4, 2, 16, 64, P, 1)):
        assert lib.attn_expand_kv4(*args, 1.0, 1.0, P, None, None) == INVALID
    assert lib.attn_expand_kv4(P, 4, 2, 16, 64, P, 1, 1.0, 1.0, ODD, None, None) == INVALID


def test_reference_quantiser_takes_the_nearest():
    """The tests' quantiser against a search over all codes and scales."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 64)) * np.exp2(rng.integers(-12, 11, size=(200, 1)))).astype(np.float32)
    bits = ref.syn.bf16_bits(x)
    x = ref.syn.bf16_to_float(bits).astype(np.float64)
    codes, scales = ref.quantise(bits, 1.0)
    for r in range(200):
        for g in range(4):
            y = x[r, g * 16:(g + 1) * 16]
            s = ref.SCALES[scales[r, g]]
            far = np.abs(ref.SCALES[:127] - np.abs(y).max() / 6)
            assert abs(s - np.abs(y).max() / 6) <= far.min() * (1 + 1e-12)
            c = codes[r, g * 8:(g + 1) * 8]
            v = ref.CODES[np.stack([c & 15, c >> 4], -1).reshape(-1)] * s
            best = np.abs(y[:, None] - ref.CODES[None, :] * s).min(1)
            assert np.all(np.abs(y - v) <= best)
