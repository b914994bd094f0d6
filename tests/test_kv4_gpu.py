"""The 4-bit KV cache on the GPU, through the library's entry points, against
plain fp64 forms (kv4_reference): the quantising append and the expansion bit
for bit, the decode within what its roundings allow.

Decode's tolerance.  The stored values and Q are used exactly.  The output is
rounded to bf16: 8 significant bits, so half a step is at most 2^-8 of a value
(just above a power of two).  P is rounded to f16: 11 significant bits, 2^-11 of
a value, and 2^-25 of one below 2^-14, where the row sum is 2^7 at least: 2^-32
of |v| a key.  Scores, exponentials and sums are fp32: (D + 4) roundings of
2^-24 of sum |q k| <= 30 here, below 2^-12 for D <= 128.  Per element: 2^-8
|out| + (2^-11 + 2^-12) sum p |v| + 2^-32 sum |v|, and for the lse 2^-12.
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from helpers import make_plan, syn

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def batch_of(qo, kv, G, Hkv, D, P, seed=0, **kw):
    return syn.make_batch("kv4", qo, kv, G * Hkv, Hkv, D, P, seed=seed, fill_pool=False, **kw)


def check_decode(batch, pool, out, lse, k_scale=1.0, v_scale=1.0, sinks="batch"):
    vals = ref.values(pool, batch.head_dim) * np.array([k_scale, v_scale])[None, :, None, None, None]
    want, want_lse, mag = ref.attention(batch, vals)
    err = np.abs(out.double().cpu().numpy() - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -32 * ref.value_sums(batch, vals) + 1e-30
    assert np.all(err <= tol), float((err / tol).max())
    if lse is not None:
        assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 2.0 ** -12


# ------------------------------------------------------------ append, expand

@pytest.mark.parametrize("Hkv,D,P,k_scale,v_scale", [(8, 64, 16, 1.0, 1.0), (2, 64, 128, 0.25, 8.0), (4, 128, 64, 2.0, 0.0625),
                                                     (1, 128, 16, 1.0, 2.0 ** -40), (3, 64, 32, 1.0, 2.0 ** 20)])
def test_append_is_exact_and_touches_nothing_else(Hkv, D, P, k_scale, v_scale):
    batch = batch_of([1, 37, 1, 0, 70], [5, 37, 300, 40, 131], 2, Hkv, D, P, seed=D + P)
    rng = np.random.default_rng(Hkv)
    k_new, v_new = syn.new_kv_rows(batch, 1)
    v_new = syn.bf16_bits(syn.bf16_to_float(v_new) * np.float32(v_scale))
    k_new[3] = 0                                                     # a row of zeros
    k_new[5, 0, 3] = 0x7F80                                          # infinity: saturates
    k_new[6, 0, 17] = 0xFFC0                                         # NaN: its group
    v_new[7, 0, :16] = syn.bf16_bits(np.float32(v_scale) * np.linspace(-2e-4, 3e-4, 16, dtype=np.float32))  # scale underflows
    v_new[8, 0, :] = syn.bf16_bits(np.float32(v_scale) * np.linspace(-9000, 9000, D, dtype=np.float32))      # saturates
    pool = rng.integers(0, 256, size=ref.pool_shape(batch.num_pages, Hkv, P, D), dtype=np.uint8)
    want = pool.copy()
    for b in range(batch.batch_size):
        for i in range(batch.qo_lens[b]):
            t, r = batch.kv_lens[b] - batch.qo_lens[b] + i, batch.qo_indptr[b] + i
            page = batch.page_table[batch.kv_indptr[b] + t // P]
            ref.put_rows(want, D, page, 0, t % P, k_new[r], k_scale)
            ref.put_rows(want, D, page, 1, t % P, v_new[r], v_scale)
    plan = make_plan(batch, dev(batch.page_table))
    got = dev(pool)
    plan.append_kv4(dev_bf16(k_new), dev_bf16(v_new), got, k_scale, v_scale)
    assert plan.device_error() == 0
    got = got.cpu().numpy()
    a, b = ref.values(got, D), ref.values(want, D)
    np.testing.assert_array_equal(np.isnan(a), np.isnan(b))
    np.testing.assert_array_equal(a[~np.isnan(a)], b[~np.isnan(b)])
    # The bytes too, but for the codes of NaN groups.
    live = ~np.isnan(b).reshape(*want.shape[:-1], 16, D // 2, 2)[..., 0].reshape(*want.shape[:-1], 8 * D)
    np.testing.assert_array_equal(got[..., :8 * D][live], want[..., :8 * D][live])
    np.testing.assert_array_equal(got[..., 8 * D:], want[..., 8 * D:])


def test_append_rounds_every_bf16_number_to_the_nearest():
    """All finite bf16 values in the range of a group whose largest is fixed, for
    every scale: borders between codes included."""
    D, P, tops = 64, 128, []
    for s in ref.SCALES[1:127]:
        tops += [6 * s, 5.9 * s, 6.2 * s]
    tops = syn.bf16_bits(np.asarray(tops, dtype=np.float32))
    rng = np.random.default_rng(0)
    rows = np.zeros((len(tops) * 4, 1, D), dtype=np.uint16)
    for i in range(len(rows)):
        top = int(tops[i // 4])
        rows[i, 0] = rng.integers(max(0, top - 0x300), top + 1, size=D) | (rng.integers(0, 2, size=D) << 15)
        rows[i, 0, ::16] = top
    # borders: (2k + 1) / 4-like multiples of each scale are bf16 numbers
    for i, s in enumerate(ref.SCALES[1:127]):
        m = np.float32(s) * np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6] * 8, dtype=np.float32)
        rows[i * 4, 0] = syn.bf16_bits(m)
    n = len(rows)
    batch = batch_of([n], [n], 1, 1, D, P)
    plan = make_plan(batch, dev(batch.page_table))
    pool = torch.zeros(plan.kv4_shape(), dtype=torch.uint8, device="cuda")
    plan.append_kv4(dev_bf16(rows), dev_bf16(rows ^ 0x8000), pool)
    want = np.zeros(pool.shape, dtype=np.uint8)
    for t in range(n):
        page = batch.page_table[t // P]
        ref.put_rows(want, D, page, 0, t % P, rows[t], 1.0)
        ref.put_rows(want, D, page, 1, t % P, rows[t] ^ 0x8000, 1.0)
    np.testing.assert_array_equal(pool.cpu().numpy(), want)


def test_append_and_expand_skip_bad_pages():
    batch = batch_of([2, 1], [40, 9], 2, 2, 64, 16, seed=9)
    rng = np.random.default_rng(1)
    pool = ref.random_pool(rng, batch.num_pages, 2, 16, 64)
    k_new, v_new = syn.new_kv_rows(batch, 0)
    pt = dev(batch.page_table)
    plan = make_plan(batch, pt)
    pt[int(batch.kv_indptr[1]) - 1] = batch.num_pages + 5
    pt[int(batch.kv_indptr[2]) - 1] = -1
    got = dev(pool)
    plan.append_kv4(dev_bf16(k_new), dev_bf16(v_new), got)
    assert plan.device_error() == 1
    assert plan.device_error() == 0
    np.testing.assert_array_equal(got.cpu().numpy(), pool)        # every new row's page is bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((3, 2, 2, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    binding().attn_expand_kv4(got, dev(np.array([1, batch.num_pages, 0], dtype=np.int32)), 64, buf=buf, device_error=err)
    assert int(err.item()) == 1
    assert torch.all(buf[1] == 7.0)
    np.testing.assert_array_equal(buf[0].double().cpu().numpy(), ref.values(pool, 64)[1])


@pytest.mark.parametrize("Hkv,D,P,n,k_scale,v_scale", [(8, 64, 16, 37, 1.0, 0.5), (1, 128, 128, 1, 2.0 ** -9, 4.0),
                                                       (5, 128, 32, 11, 1.0, 1.0), (2, 64, 64, 600, 2.0 ** 40, 2.0 ** -40)])
def test_expand_is_exact(Hkv, D, P, n, k_scale, v_scale):
    rng = np.random.default_rng(n)
    pool = rng.integers(0, 256, size=ref.pool_shape(n + 3, Hkv, P, D), dtype=np.uint8)   # every scale byte, NaN and signs
    ids = rng.permutation(n + 3)[:n].astype(np.int32)
    ids[-1] = ids[0]                                                                     # a page twice
    got = binding().attn_expand_kv4(dev(pool), dev(ids), D, k_scale=k_scale, v_scale=v_scale).double().cpu().numpy()
    want = ref.values(pool, D)[ids] * np.array([k_scale, v_scale])[None, :, None, None, None]
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


# -------------------------------------------------------------------- decode

@pytest.mark.parametrize("G", [1, 3, 8, 9, 16, 20])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (64, 128), (128, 16)])
def test_decode_matches_reference(G, D, P):
    kv = [1, 15, 16, 17, 33, 100, 257, 1, 600]
    batch = batch_of([1] * len(kv), kv, G, 2, D, P, seed=G + D, with_sinks=G % 2 == 0)
    rng = np.random.default_rng(G * D)
    pool = ref.random_pool(rng, batch.num_pages, 2, P, D)
    ref.poison_unused(pool, batch)
    plan = make_plan(batch, dev(batch.page_table))
    q = dev_bf16(batch.q)
    sinks = None if batch.sinks is None else dev(batch.sinks)
    lse = torch.empty(batch.total_rows, batch.num_qo_heads, device="cuda")
    out, _ = plan.decode_kv4(q, dev(pool), sinks, lse=lse)
    assert plan.device_error() == 0
    check_decode(batch, pool, out, lse)


@pytest.mark.parametrize("D,P,num_sms", [(64, 16, 0), (128, 64, 0), (64, 32, 1)])
def test_decode_split_sequences(D, P, num_sms):
    """Long sequences split over CTAs, with the pool's scales and without an lse."""
    kv = [5000, 129, 2049]
    batch = batch_of([1] * 3, kv, 8, 1, D, P, seed=D)
    pool = ref.random_pool(np.random.default_rng(P), batch.num_pages, 1, P, D)
    ref.poison_unused(pool, batch)
    plan = make_plan(batch, dev(batch.page_table), num_sms=num_sms)
    if num_sms == 0:
        assert plan.info()["num_decode_groups_split"] > 0
    q, d_pool, sinks = dev_bf16(batch.q), dev(pool), dev(batch.sinks)
    lse = torch.empty(3, 8, device="cuda")
    out, _ = plan.decode_kv4(q, d_pool, sinks, lse=lse, k_scale=0.5, v_scale=4.0)
    check_decode(batch, pool, out, lse, 0.5, 4.0)
    again, none = plan.decode_kv4(q, d_pool, sinks, k_scale=0.5, v_scale=4.0)     # counters are ready again; same bits
    assert none is None and torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert plan.device_error() == 0


def test_decode_very_low_scores():
    """All scores far below zero: the softmax shift follows them down, in every
    warp, also in those that have no tokens; and rows whose scores rise or fall
    by hundreds along the sequence."""
    batch = batch_of([1, 1, 1], [33, 700, 700], 8, 1, 64, 16, seed=13, with_sinks=False)
    rng = np.random.default_rng(1)
    pool = ref.random_pool(rng, batch.num_pages, 1, 16, 64, spread=0.3)
    codes = pool[..., :8 * 64]
    codes[:, 0] = (codes[:, 0] & 0x77) | 0x00                      # K positive
    q = np.abs(syn.bf16_to_float(batch.q))
    q[0] *= -40                                                    # scores around -700
    batch.q = syn.bf16_bits(q)
    t = np.arange(700)
    for b, up in ((1, 1), (2, -1)):
        page = batch.page_table[batch.kv_indptr[b] + t // 16]
        level = (20 + t * 50 // 700) if up > 0 else (70 - t * 50 // 700)
        for k in range(4):
            pool[page, 0, :, 0, 8 * 64 + (t % 16) * 4 + k] = level[:, None].astype(np.uint8)
    ref.poison_unused(pool, batch)
    plan = make_plan(batch, dev(batch.page_table))
    lse = torch.empty(3, 8, device="cuda")
    out, _ = plan.decode_kv4(dev_bf16(batch.q), dev(pool), lse=lse)
    vals = ref.values(pool, 64)
    want, want_lse, mag = ref.attention(batch, vals)
    qf = syn.bf16_to_float(batch.q).astype(np.float64)
    # 68 roundings of 2^-24 of sum |q k| in the exponent (all products have one sign here).
    size = np.stack([np.abs(ref.gather(batch, vals, b, 0)[0] @ qf[b].T).max(0) for b in range(3)]) / 8
    slack = 68 * 2.0 ** -24 * size
    err = np.abs(out.double().cpu().numpy() - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12 + 2 * slack[..., None]) * mag + \
        2.0 ** -32 * ref.value_sums(batch, vals) + 1e-30
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -12 + slack + 2.0 ** -22 * np.abs(want_lse))


def test_decode_nan_stays_in_its_request_and_head():
    """A NaN scale among a request's keys or values reaches that request's heads
    of that KV head (for V, the 16 dims) and nothing else."""
    batch = batch_of([1, 1], [100, 90], 4, 2, 64, 16, seed=17)
    pool = ref.random_pool(np.random.default_rng(6), batch.num_pages, 2, 16, 64)
    clean = pool.copy()
    p0 = batch.page_table[batch.kv_indptr[0]]
    pool[p0, 0, 0, 0, 8 * 64 + 5] = 0x7F                            # a K scale of head 0
    pool[p0, 1, 1, 0, 8 * 64 + 4 * 3 + 2] = 0x7F                    # a V scale of head 1: dims 32..47
    plan = make_plan(batch, dev(batch.page_table))
    a, _ = plan.decode_kv4(dev_bf16(batch.q), dev(pool), dev(batch.sinks))
    b, _ = plan.decode_kv4(dev_bf16(batch.q), dev(clean), dev(batch.sinks))
    bad = torch.isnan(a)
    assert torch.all(bad[0, :4]) and torch.all(bad[0, 4:, 32:48])
    bad[0, :4], bad[0, 4:, 32:48] = False, False
    assert not torch.any(bad)
    same = torch.ones_like(bad)
    same[0, :4], same[0, 4:, 32:48] = False, False
    assert torch.equal(a[same], b[same])


def test_decode_large_scores_and_sinks():
    """Scores that grow along the sequence (the running max moves again and
    again), sinks above and below everything, and heads of very different size."""
    batch = batch_of([1, 1], [700, 64], 8, 2, 64, 16, seed=3)
    pool = ref.random_pool(np.random.default_rng(4), batch.num_pages, 2, 16, 64, spread=0.5)
    t = np.arange(700)
    page = batch.page_table[batch.kv_indptr[0] + t // 16]
    for k in range(4):   # K's scales rise with the position
        pool[page, 0, :, 0, 8 * 64 + (t % 16) * 4 + k] = (20 + t * 60 // 700)[:, None].astype(np.uint8)
    q = syn.bf16_to_float(batch.q)
    q[:, 0] *= 2.0 ** 20
    pool[page, 0, :, 0, 8 * 64:] = np.minimum(pool[page, 0, :, 0, 8 * 64:], 70)
    q[:, 0] /= 2.0 ** 18
    q[:, 1] *= 2.0 ** -30
    q[:, 2] = 0
    batch.q = syn.bf16_bits(q)
    batch.sinks = np.array([-50, 60, 0, 1, -np.inf, 2, 3, 88] * 2, dtype=np.float32)
    plan = make_plan(batch, dev(batch.page_table))
    lse = torch.empty(2, 16, device="cuda")
    out, _ = plan.decode_kv4(dev_bf16(batch.q), dev(pool), dev(batch.sinks), lse=lse)
    vals = ref.values(pool, 64)
    with np.errstate(divide="ignore"):
        want, want_lse, mag = ref.attention(batch, vals)
    err = np.abs(out.double().cpu().numpy() - want)
    # sum |q k| reaches 300 here: (D + 4) 2^-24 of it is 2^-9.7 in the exponent.
    size = max(np.abs(ref.gather(batch, vals, b, 0)[h // 8] @ q[b, h]).max() for b in range(2) for h in range(16)) / 8
    slack = 68 * 2.0 ** -24 * 4 * size
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12 + 2 * slack) * mag +
                  2.0 ** -32 * ref.value_sums(batch, vals) + 1e-30)
    assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 2.0 ** -12 + slack + 2.0 ** -22 * np.abs(want_lse).max()


def test_decode_leaves_other_rows_alone_and_skips_bad_pages():
    batch = batch_of([1, 3, 0, 1], [20, 30, 12, 200], 4, 2, 64, 16, seed=6)
    pool = ref.random_pool(np.random.default_rng(5), batch.num_pages, 2, 16, 64)
    pt = dev(batch.page_table)
    plan = make_plan(batch, pt)
    out = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 8), 3.0, device="cuda")
    plan.decode_kv4(dev_bf16(batch.q), dev(pool), dev(batch.sinks), out, lse)
    assert torch.all(out[1:4] == 3.0) and torch.all(lse[1:4] == 3.0)      # prefill rows
    good = out[4].clone()
    pt[0] = -3
    plan.decode_kv4(dev_bf16(batch.q), dev(pool), dev(batch.sinks), out, lse)
    assert plan.device_error() == 1
    assert torch.equal(out[4], good)


def test_empty_batches():
    b = binding()
    pt = torch.zeros(0, dtype=torch.int32, device="cuda")
    plan = b.Plan([0], [0], pt, [], 8, 2, 64, 16, num_pages=4)
    q = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(plan.kv4_shape(), dtype=torch.uint8, device="cuda")
    w = torch.zeros(4, 2, 16, device="cuda")
    plan.append_kv4(kv, kv, pool)
    plan.decode_kv4(q, pool)
    plan.key_weights_kv4(q, pool, torch.empty(0, 8, device="cuda"), w)
    assert plan.evict_kv4(w, pool, 5, 2).shape == (0, 2, 5)
    assert b.attn_expand_kv4(pool, pt, 64).shape == (0, 2, 2, 16, 64)
    assert plan.device_error() == 0


def test_prefill_over_an_expanded_cache():
    """A chunk appended in 4 bits, its request's pages expanded, and the bf16
    prefill over them: what a chunked prefill on a 4-bit cache does."""
    from helpers import check_close
    batch = batch_of([70, 33], [200, 33], 4, 2, 64, 16, seed=12)
    pool = ref.random_pool(np.random.default_rng(2), batch.num_pages, 2, 16, 64)
    k_new, v_new = syn.new_kv_rows(batch, 5)
    pt = dev(batch.page_table)
    plan = make_plan(batch, pt)
    d_pool = dev(pool)
    plan.append_kv4(dev_bf16(k_new), dev_bf16(v_new), d_pool)
    bf16_pool = binding().attn_expand_kv4(d_pool, pt, 64)
    n = pt.numel()
    work = binding().Plan(batch.qo_indptr, batch.kv_indptr, torch.arange(n, dtype=torch.int32, device="cuda"),
                          batch.last_page_len, 8, 2, 64, 16, num_pages=n)
    lse = torch.empty(batch.total_rows, 8, device="cuda")
    out, _ = work.prefill(dev_bf16(batch.q), bf16_pool, dev(batch.sinks), lse=lse)
    want, want_lse, _ = ref.attention(batch, ref.values(d_pool.cpu().numpy(), 64))
    check_close(out, lse, want, want_lse, "prefill over an expanded cache")


def test_refusals():
    b = binding()
    batch = batch_of([1, 1], [20, 30], 4, 2, 64, 16)
    pool = ref.random_pool(np.random.default_rng(0), batch.num_pages, 2, 16, 64)
    plan = make_plan(batch, dev(batch.page_table))
    q, p = dev_bf16(batch.q), dev(pool)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (0.0, -1.0, 3.0, float("inf"), float("nan"), 2.0 ** 41, 2.0 ** -41):
        with pytest.raises(b.AttnError):
            plan.decode_kv4(q, p, k_scale=bad)
        with pytest.raises(b.AttnError):
            plan.append_kv4(kv, kv, p, v_scale=bad)
        with pytest.raises(b.AttnError):
            b.attn_expand_kv4(p, torch.zeros(1, dtype=torch.int32, device="cuda"), 64, v_scale=bad)
    with pytest.raises(ValueError):
        plan.decode_kv4(q, p[:-1])
    with pytest.raises(TypeError):
        plan.decode_kv4(q.float(), p)
    with pytest.raises(TypeError):
        plan.decode_kv4(q, p.cpu())
    with pytest.raises(TypeError):
        plan.append_kv4(kv.transpose(0, 1), kv, p)
    with pytest.raises(ValueError):
        b.attn_expand_kv4(p, torch.zeros(1, dtype=torch.int32, device="cuda"), 128)
    ragged = b.RaggedPlan([0, 4], [0, 4], 8, 2, 64)
    with pytest.raises(TypeError):
        ragged.decode_kv4(q, p)
    graph = b.GraphPlan(2, 8, 2, 64, 16, plan.page_table, batch.num_pages)
    with pytest.raises(TypeError):
        graph.decode_kv4(q, p)
    assert b.kv4_cache_shape(3, 2, 32, 128) == (3, 2, 2, 2, 1152)
    with pytest.raises(ValueError):
        b.kv4_cache_shape(3, 2, 24, 128)
