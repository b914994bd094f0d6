"""CPU checks of cross attention's planner and entry points: what is refused, and
that the planned work covers every (row, head) pair and key exactly once."""
import ctypes

import numpy as np
import pytest

from test_abi import FAKE_PT, INVALID, OK, UNSUPPORTED, lib, units_of   # noqa: F401  (lib: the built library's fixture)

P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
NOT_BOUND = 5


def plan(lib, qo, start, lens, kv_rows, Hq=8, Hkv=2, D=64, scale=0.125, sms=152, batch=None, null=()):
    arrays = [np.concatenate([[0], np.cumsum(qo)]).astype(np.int32), np.asarray(start, np.int32), np.asarray(lens, np.int32)]
    args = [None if i in null else a.ctypes.data for i, a in enumerate(arrays)]
    h, ws = ctypes.c_void_p(), ctypes.c_size_t()
    st = lib.attn_plan_cross(*args, len(qo) if batch is None else batch, kv_rows, Hq, Hkv, D, scale, sms, ctypes.byref(h),
                             ctypes.byref(ws))
    return st, h, ws.value


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), INVALID), (dict(kv_rows=-1), INVALID), (dict(kv_rows=9), INVALID), (dict(start=[-1]), INVALID),
    (dict(lens=[-1]), INVALID), (dict(start=[2 ** 31 - 1]), INVALID), (dict(qo=[-1]), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID), (dict(D=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(sms=-1), INVALID), (dict(null=(0,)), INVALID),
    (dict(null=(1,)), INVALID), (dict(null=(2,)), INVALID), (dict(qo=[2 ** 28]), UNSUPPORTED),
    (dict(kv_rows=2 ** 30 + 5), UNSUPPORTED)])
def test_bad_plans(lib, bad, status):
    st, h, _ = plan(lib, **{**dict(qo=[3], start=[2], lens=[8], kv_rows=10), **bad})
    assert st == status and not h.value


def test_null_results(lib):
    ind = np.zeros(2, np.int32)
    assert lib.attn_plan_cross(ind.ctypes.data, ind.ctypes.data, ind.ctypes.data, 1, 0, 8, 2, 64, 0.125, 152, None, None) == INVALID


def cross(lib, h, q=P, k=P, ks=128, v=P, vs=128, sinks=P, out=P, lse=P):
    return lib.attn_cross(h, q, k, ks, v, vs, sinks, out, lse, None)


def test_launches_are_refused_before_the_device(lib):
    st, h, _ = plan(lib, [3], [0], [8], 8)
    assert st == OK and cross(lib, h) == NOT_BOUND and cross(lib, None) == INVALID
    # Every other launch, and a cross launch of another plan.
    p = lambda n: [P] * n
    assert lib.attn_decode(h, *p(5), None) == INVALID
    assert lib.attn_decode_noalloc(h, *p(5), None) == INVALID
    assert lib.attn_prefill(h, *p(5), None) == INVALID
    assert lib.attn_prefill_ragged(h, *p(6), None) == INVALID
    assert lib.attn_append_kv(h, *p(3), None) == INVALID
    assert lib.attn_decode_kv4(h, P, P, 1.0, 1.0, None, P, None, None) == INVALID
    assert lib.attn_key_weights(h, P, P, P, P, 1.0, 0, P, None) == INVALID
    assert lib.attn_evict_kv(h, P, P, 4, 1, P, P, 10, P, P, None) == INVALID
    assert lib.attn_plan_get_kv_lens(h, P, 0) == INVALID
    lib.attn_plan_destroy(h)
    r, ws = ctypes.c_void_p(), ctypes.c_size_t()
    ind = np.array([0, 4], dtype=np.int32)
    assert lib.attn_plan_ragged(ind.ctypes.data, ind.ctypes.data, 1, 8, 2, 64, 1, 0.125, 152, ctypes.byref(r),
                                ctypes.byref(ws)) == OK
    assert cross(lib, r) == INVALID
    lib.attn_plan_destroy(r)


def test_the_binding_refuses_the_other_calls():
    from paged_kv_attention_sink_gb300 import binding
    empty = object.__new__(binding.CrossPlan)
    for name in ("decode", "prefill", "append_kv", "append_kv_rope", "append_kv4", "decode_kv4", "key_weights",
                 "key_weights_kv4", "evict_kv", "evict_kv4", "kv4_shape"):
        with pytest.raises(TypeError):
            getattr(empty, name)()
    with pytest.raises(TypeError):
        empty.kv_lens
    with pytest.raises(ValueError):
        binding.CrossPlan([0, 1], [0, 0], [1, 1], 4, 8, 2, 64)
    for bad in (dict(kv_rows=2 ** 31), dict(kv_rows=-1), dict(kv_start=[2 ** 32]), dict(kv_len=[2 ** 31])):
        with pytest.raises(ValueError):
            binding.CrossPlan(**{**dict(qo_indptr=[0, 1], kv_start=[0], kv_len=[1], kv_rows=4, num_qo_heads=8, num_kv_heads=2,
                                        head_dim=64), **bad})


@pytest.mark.parametrize("sms", [152, 4])
@pytest.mark.parametrize("Hq,Hkv,D,seed", [(8, 2, 64, 0), (16, 16, 64, 1), (64, 4, 128, 2), (20, 4, 64, 3), (9, 3, 128, 4),
                                           (160, 1, 64, 5), (128, 1, 128, 6), (64, 8, 64, 7), (7, 1, 64, 8)])
def test_every_pair_and_key_once(lib, Hq, Hkv, D, seed, sms):
    rng = np.random.default_rng(seed)
    G = Hq // Hkv
    qo = [0, 1, 1, 3, 16 // min(G, 16), 64 // min(G, 64) + 1, 200, 700, int(rng.integers(1, 40)), 5, 64]
    kv = [9, 0, 1, 64, 65, 5000, 129, 1500, 40000, 0, 640]
    start = [int(rng.integers(0, 100)) for _ in kv]
    st, h, _ = plan(lib, qo, start, kv, 45000, Hq, Hkv, D, sms=sms)
    assert st == OK
    info, units, items = units_of(lib, h)
    ind = np.concatenate([[0], np.cumsum(qo)])
    seen = {}                                                       # (sequence, KV head, pair) -> key ranges

    def add(b, g, pairs, t0, t1, chunk):
        for p in pairs:
            seen.setdefault((b, g, p), []).append((t0, t1, chunk))

    slots, merges = set(), 0
    for q_row, first, g, p0, n, t0, t1, chunk, n_chunks, group, partial0, shared in units.tolist():
        b = int(np.searchsorted(ind, q_row, "right")) - 1
        assert q_row == ind[b] and first == start[b] and 1 <= n <= 32 and 0 <= t0 <= t1 <= kv[b]
        assert t0 % 64 == 0 and (t1 % 64 == 0 or t1 == kv[b]) and shared == (qo[b] * G > 32)
        add(b, g, range(p0, p0 + n), t0, t1, (chunk, n_chunks))
        tiles = 1 if n <= 16 else 2
        for s in range(tiles if n_chunks > 1 else 0):
            slot = partial0 + chunk * tiles + s
            assert 0 <= slot < info.num_decode_partials and slot not in slots
            slots.add(slot)
        merges += (n_chunks > 1 and chunk == 0)
    sizes = [1 if n <= 16 else 2 for n in units[:, 4]]
    assert sizes == sorted(sizes)
    rows = 128 // min(G, 128)
    chunks = {}
    for q_row0, n0, first, kv_len, partial, g, head0, n_slots, tiles, key_end, n1, c in items.tolist():
        chunks[q_row0, g] = max(chunks.get((q_row0, g), 0), c + 1)
    for q_row0, n0, first, kv_len, partial, g, head0, n_slots, tiles, key_end, n1, c in items.tolist():
        b = int(np.searchsorted(ind, q_row0, "right")) - 1
        t0 = first - start[b]
        assert t0 % 128 == 0 and kv_len == key_end > 0 and tiles == -(-kv_len // 128) and head0 == g * G
        assert (partial >= 0) == (chunks[q_row0, g] > 1)
        for s in range(8 * n_slots if partial >= 0 else 0):
            assert 0 <= partial + s < info.num_decode_partials and partial + s not in slots
            slots.add(partial + s)
        merges += (-(-n0 // 32) - (-n1 // 32)) * (partial >= 0 and c == 0)
        assert n_slots == (2 if n1 else 1) and 0 < n0 <= 128 and n1 <= 128 and (not n1 or n0 == rows * G)
        p0 = (q_row0 - int(ind[b])) * G
        add(b, g, range(p0, p0 + n0 + n1), t0, t0 + kv_len, (c, chunks[q_row0, g]))
    assert len(slots) == info.num_decode_partials and merges == info.num_decode_groups_split
    for b in range(len(qo)):
        for g in range(Hkv):
            for p in range(qo[b] * G):
                parts = sorted(seen.pop((b, g, p)))
                assert parts[0][0] == 0 and parts[-1][1] == kv[b]
                assert all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
                assert [x[2] for x in parts] == [(c, len(parts)) for c in range(len(parts))]
    assert not seen
    lib.attn_plan_destroy(h)


def test_one_long_sequence_among_many_short_ones_is_split(lib):
    """No item or unit is much longer than an even share of the work."""
    for rows in (40, 3):                                           # the prefill kernel's, and few rows
        qo, kv = [rows] * 800, [200] * 799 + [600000]
        start = [0] * 800
        st, h, _ = plan(lib, qo, start, kv, 600000)
        assert st == OK
        _, units, items = units_of(lib, h)
        if rows == 40:
            share = items[:, 8].sum() / 152
            assert len(units) == 0 and items[:, 8].max() <= 1.5 * share + 1
        else:
            lens = (units[:, 6] - units[:, 5] + 63) // 64
            assert len(items) == 0 and lens.max() <= 1.5 * lens.sum() / (3 * 152) + 4
        lib.attn_plan_destroy(h)
