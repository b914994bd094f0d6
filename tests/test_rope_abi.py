"""CPU checks of the rotary entry points: arguments are refused with a status
before anything reaches the device (the pointers here are never dereferenced),
and the reference's angles are checked against each other."""
import ctypes
import math

import numpy as np
import pytest

import rope_reference as ref
from test_abi import INVALID, OK, UNSUPPORTED, lib, plan   # noqa: F401  (lib: the built library's fixture)

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
NOT_BOUND = 5


class Spec:
    """An attn_rope_spec that keeps its arrays."""

    def __init__(self, rot=64, interleaved=0, n_axes=1, scale=1.0, freq=None, axis=None):
        from paged_kv_attention_sink_gb300.binding import RopeSpec
        n = max(1, rot // 2)
        self.freq = np.full(n, 0.5, np.float32) if freq is None else np.asarray(freq, np.float32)
        self.axis = None if axis is None else np.asarray(axis, np.int32)
        self.c = RopeSpec(rot, interleaved, n_axes, scale, self.freq.ctypes.data, self.axis.ctypes.data if axis is not None else None)

    @property
    def p(self):
        return ctypes.addressof(self.c)


def rope(lib, spec, positions=P, rows=4, D=64, q=P, qs=512, Hq=8, qo=P, qos=512, k=P, ks=128, Hk=2, ko=P, kos=128, inverse=0):
    return lib.attn_rope(spec.p if spec else None, positions, rows, D, q, qs, Hq, qo, qos, k, ks, Hk, ko, kos, inverse, None)


def test_rows_of_none_are_fine(lib):
    assert rope(lib, Spec(), rows=0) == OK
    assert rope(lib, Spec(), rows=0, q=None, k=None, qo=None, ko=None, positions=None) == OK


@pytest.mark.parametrize("spec", [dict(rot=0), dict(rot=80), dict(interleaved=2), dict(n_axes=0), dict(n_axes=9),
                                  dict(scale=float("nan")), dict(scale=float("inf")), dict(freq=[float("nan")] * 32),
                                  dict(freq=[2.0 ** 20] * 32), dict(freq=[-(2.0 ** 20)] * 32), dict(axis=[1] * 32),
                                  dict(axis=[-1] * 32, n_axes=2)])
def test_bad_specs(lib, spec):
    assert rope(lib, Spec(**spec), rows=0) == INVALID


def test_null_and_unsupported_specs(lib):
    assert rope(lib, None) == INVALID
    empty = Spec()
    empty.c.inv_freq = None
    assert rope(lib, empty) == INVALID
    assert rope(lib, Spec(rot=24)) == UNSUPPORTED
    assert rope(lib, Spec(), D=96, qs=768, qos=768, ks=192, kos=192) == UNSUPPORTED
    assert rope(lib, Spec(), rows=1 << 31) == UNSUPPORTED
    assert rope(lib, Spec(), Hq=65535, Hk=2) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(Hq=-1), dict(Hk=-1), dict(Hq=0, Hk=0), dict(inverse=2), dict(positions=None),
                                 dict(positions=ctypes.c_void_p(0x10002)), dict(q=None), dict(qo=None), dict(k=None),
                                 dict(ko=None), dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(ko=ODD), dict(qs=511),
                                 dict(qs=516), dict(qos=504), dict(ks=120), dict(kos=132), dict(qs=1024), dict(ks=1024)])
def test_bad_arguments(lib, bad):
    assert rope(lib, Spec(), **bad) == INVALID        # (the last two: in place with another stride)


def test_append(lib):
    st, h, _ = plan(lib, [1], [2], [4])
    call = lambda h, spec=Spec(): lib.attn_append_kv_rope(h, spec.p, P, P, 16 * 64, P, 128, P, 128, P, P, None)
    assert call(None) == INVALID and call(h) == NOT_BOUND
    lib.attn_plan_destroy(h)
    r, g, ws = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_size_t()
    ind = np.array([0, 4], dtype=np.int32)
    assert lib.attn_plan_ragged(ind.ctypes.data, ind.ctypes.data, 1, 16, 2, 64, 1, 0.125, 152, ctypes.byref(r),
                                ctypes.byref(ws)) == OK
    assert lib.attn_graph_plan(8, 16, 2, 64, 16, ctypes.c_float(0.125), 1024, 8 * 4096, P, 152, ctypes.byref(g),
                               ctypes.byref(ws)) == OK
    for other in (r, g):
        assert call(other) == INVALID
        lib.attn_plan_destroy(other)


def test_the_binding_refuses_without_a_device():
    from paged_kv_attention_sink_gb300 import binding
    with pytest.raises(ValueError):
        binding.Rope([])
    with pytest.raises(ValueError):
        binding.Rope([1.0, 0.5], axis=[0])
    with pytest.raises(ValueError):
        binding.Rope([1.0, 0.5], axis=[0, -1])
    with pytest.raises(TypeError):
        binding.Rope([1.0] * 8).apply(None, np.zeros((1, 1, 64)))
    for kind in ("RaggedPlan", "GraphPlan"):
        with pytest.raises(TypeError):
            object.__new__(getattr(binding, kind)).append_kv_rope()


@pytest.mark.parametrize("pos,freq", [(0, 1.0), (1, 1.0), (-1, 1.0), (4097, 0.25), (1 << 20, 1e-4), (100003, 0.7)])
def test_the_references_angles(pos, freq):
    """Where 64-bit floats still hold the angle, both ways agree (a rounding of pos * freq: 2^-53 of it)."""
    f = float(np.float32(freq))
    t = ref.turn_fraction(pos, freq)
    assert abs(math.cos(2 * math.pi * t) - math.cos(pos * f)) <= 2.0 ** -50 * (1 + abs(pos * f))
    assert abs(math.sin(2 * math.pi * t) - math.sin(pos * f)) <= 2.0 ** -50 * (1 + abs(pos * f))
