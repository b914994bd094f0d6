"""Cross attention on the GPU against the plain 64-bit form.

Tolerance.  P is rounded to bf16, by at most 2^-8 of a weight, and O normalised by
the sum of that rounded P, which is off by as much at most: (1 + 2^-8) / (1 - 2^-8)
- 1 < 2^-7 + 2^-13 of sum w |v|.  The output's own rounding is half a step, 2^-8 of
the value.  Scores, exponentials and sums are fp32: (D + 4) roundings of 2^-24 of
scale sum |q k| <= 60 here, and ex2.approx and the merge's 2^-22 each: below 2^-11
for D <= 128, relative in a weight and absolute in the lse.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def inputs(qo, kv, Hq, Hkv, D, sinks, padded=True, fused=True, seed=0, big=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    room = max(kv) + 3
    start = [b * room + 1 for b in range(len(kv))] if padded else np.concatenate([[0], np.cumsum(kv)[:-1]]).tolist()
    rows = room * len(kv) + 1 if padded else sum(kv)
    both = torch.randn(rows, 2 * Hkv, D, device="cuda", generator=g).to(torch.bfloat16)
    if padded:
        keep = torch.zeros(rows, dtype=torch.bool)
        for s, n in zip(start, kv):
            keep[s:s + n] = True
        both[~keep.cuda()] = float("nan")
    k, v = both[:, :Hkv], both[:, Hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    q = (big * torch.randn(sum(qo), Hq, D, device="cuda", generator=g)).to(torch.bfloat16)
    s = torch.randn(Hq, device="cuda", generator=g) if sinks else None
    return q, k, v, s, start, rows


def plain(q, k, v, s, qo, start, kv, scale):
    Hq, Hkv = q.shape[1], k.shape[1]
    out, mag, lse, r0 = [], [], [], 0
    for n, st, m in zip(qo, start, kv):
        x, kk, vv = q[r0:r0 + n].double(), k[st:st + m].double(), v[st:st + m].double()
        r0 += n
        kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (kk, vv))
        sc = torch.einsum("rhd,thd->rht", x, kk) * scale
        z = sc if s is None else torch.cat((sc, s.double()[None, :, None].expand(n, -1, 1)), -1)
        if z.shape[-1] == 0:
            out.append(torch.zeros_like(x))
            mag.append(torch.zeros_like(x))
            lse.append(torch.full((n, Hq), -float("inf"), dtype=torch.float64, device=q.device))
            continue
        le = torch.logsumexp(z, -1)
        w = torch.exp(sc - le[..., None])
        out.append(torch.einsum("rht,thd->rhd", w, vv))
        mag.append(torch.einsum("rht,thd->rhd", w, vv.abs()))
        lse.append(le)
    return torch.cat(out), torch.cat(mag), torch.cat(lse)


def check(qo, kv, Hq, Hkv, D, sinks, scale=None, num_sms=0, **kw):
    q, k, v, s, start, rows = inputs(qo, kv, Hq, Hkv, D, sinks, **kw)
    scale = D ** -0.5 if scale is None else scale
    plan = binding().CrossPlan(np.concatenate([[0], np.cumsum(qo)]), start, kv, rows, Hq, Hkv, D, sm_scale=scale,
                               num_sms=num_sms)
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    plan.attend(q, k, v, s, out, lse)
    assert plan.device_error() == 0
    want, mag, want_lse = plain(q, k, v, s, qo, start, kv, scale)
    err = (out.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -13 + 2.0 ** -11) * mag + 1e-30
    assert bool((err <= tol).all()), float((err / tol).nan_to_num(1e9).max())
    same = torch.isinf(want_lse)
    assert torch.equal(lse.double()[same], want_lse[same])
    assert bool(((lse.double() - want_lse)[~same].abs() <= 2.0 ** -11).all())
    # The same again, without lse, into fresh memory: the order of every sum is fixed.
    again, _ = plan.attend(q, k, v, s)
    assert torch.equal(again, out)
    return plan, (q, k, v, s), out, lse


HEADS = [(1, 1, 64), (8, 2, 64), (16, 16, 128), (64, 8, 64), (64, 4, 128), (15, 5, 64), (12, 1, 128), (40, 8, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("sinks", [False, True])
def test_single_rows(Hq, Hkv, D, sinks):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 128, 300, 1500]
    plan, *_ = check([1] * len(kv), kv, Hq, Hkv, D, sinks, seed=Hq + D)
    assert plan.info()["num_prefill_items"] == 0


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("padded,fused,sms", [(True, True, 3), (False, False, 20), (True, False, 0)])
def test_rows_of_every_number(Hq, Hkv, D, padded, fused, sms):
    """Blocks of one and two tiles, the border to the prefill kernel, several blocks and slots; no rows, no keys."""
    qo = [2, 3, 0, 5, 8, 11, 16, 17, 33, 63, 64, 65, 127, 129, 260, 4, 30]
    kv = [70, 16, 9, 33, 64, 65, 129, 1, 128, 200, 257, 64, 300, 127, 500, 0, 0]
    plan, *_ = check(qo, kv, Hq, Hkv, D, True, padded=padded, fused=fused, seed=D, num_sms=sms)
    info = plan.info()
    assert info["num_decode_units"] > 0 and (sms != 3 or info["num_prefill_items"] > 0)


@pytest.mark.parametrize("Hq,Hkv,D,qo", [(8, 2, 64, 3), (64, 4, 128, 1), (16, 16, 64, 5), (4, 1, 64, 16), (6, 2, 128, 11)])
def test_long_keys_are_split(Hq, Hkv, D, qo):
    plan, *_ = check([qo, qo, 1], [20000, 2999, 70001], Hq, Hkv, D, True, seed=qo)
    assert plan.info()["num_decode_partials"] > 0


@pytest.mark.parametrize("Hq,Hkv,D,qo", [(8, 2, 64, 20), (4, 4, 128, 300), (64, 8, 64, 5), (10, 2, 64, 97), (6, 1, 128, 22),
                                          (48, 1, 64, 3), (130, 1, 128, 2)])
def test_many_rows_over_split_keys(Hq, Hkv, D, qo):
    plan, *_ = check([qo, qo, 1, qo], [5000, 700, 9000, 1153], Hq, Hkv, D, qo % 2 == 0, seed=qo, num_sms=12)
    info = plan.info()
    assert info["num_decode_partials"] > 0 and (Hq // Hkv > 128 or info["num_prefill_items"] > 2 * Hkv)
    check([qo, qo, 1, qo], [5000, 700, 9000, 1153], Hq, Hkv, D, qo % 2 == 1, seed=qo)


@pytest.mark.parametrize("Hq,Hkv,D,qo,kv", [(8, 1, 64, 1, 1000003), (2, 1, 128, 150, 200003), (2, 2, 64, 12, 300001)])
def test_very_long_keys(Hq, Hkv, D, qo, kv):
    check([qo], [kv], Hq, Hkv, D, True, seed=1, padded=False)


def test_states_past_4_gb():
    """Rows whose offsets pass 32 bits, in bytes and in elements."""
    rows, Hkv, D = 300000, 64, 128
    both = torch.empty(rows, 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")       # 9.8 GB
    g = torch.Generator(device="cuda").manual_seed(3)
    start, kv = [0, rows - 1000, rows - 77], [100, 900, 77]
    for s, n in zip(start, kv):
        both[s:s + n] = torch.randn(n, 2 * Hkv, D, device="cuda", generator=g).to(torch.bfloat16)
    k, v = both[:, :Hkv], both[:, Hkv:]
    qo = [2, 70, 1]
    q = torch.randn(sum(qo), Hkv, D, device="cuda", generator=g).to(torch.bfloat16)
    plan = binding().CrossPlan(np.concatenate([[0], np.cumsum(qo)]), start, kv, rows, Hkv, Hkv, D)
    out, _ = plan.attend(q, k, v)
    want, mag, _ = plain(q, k, v, None, qo, start, kv, D ** -0.5)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -10) * mag).all())


@pytest.mark.parametrize("D", [64, 128])
def test_kernels_beside_one_another_follow_what_came_before_and_are_followed(D):
    """Calls that feed one another: each reads the last one's output as queries, on one stream, many times over, and
    the same with every kernel of the first waiting for a late one."""
    qo, kv = [1, 9, 40, 3, 100, 7], [3000, 700, 2000, 65, 900, 5000]
    plan, (q, k, v, s), *_ = check(qo, kv, 8, 2, D, False, seed=30, num_sms=10)
    info = plan.info()
    assert info["num_prefill_items"] and info["num_decode_units"] and info["num_decode_partials"]
    x = q.clone()
    want = []
    for _ in range(4):
        x = plan.attend(x, k, v)[0]
        torch.cuda.synchronize()
        want.append(x.clone())
    buf = [torch.empty_like(q), torch.empty_like(q)]
    for _ in range(20):
        buf[0].copy_(q)
        for i in range(4):
            plan.attend(buf[i % 2], k, v, out=buf[(i + 1) % 2])
        assert torch.equal(buf[0], want[-1])
        torch.cuda._sleep(20000)
        buf[0].zero_().add_(q)
        for i in range(3):
            plan.attend(buf[i % 2], k, v, out=buf[(i + 1) % 2])
        assert torch.equal(buf[1], want[2])


def test_two_plans_at_once():
    """Each with its own workspace, on its own stream."""
    cases = [([3, 200, 1], [9000, 700, 4000]), ([5, 64, 2, 90], [1500, 3000, 64, 5000])]
    made = [check(qo, kv, 16, 4, 64, True, seed=20 + i) for i, (qo, kv) in enumerate(cases)]
    streams, outs = [torch.cuda.Stream() for _ in made], []
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [plan.attend(*x, stream=s)[0] for (plan, x, _, _), s in zip(made, streams)]
    torch.cuda.synchronize()
    for out, (plan, _, want, _) in zip(outs, made):
        assert torch.equal(out, want) and plan.device_error() == 0


@pytest.mark.parametrize("G,D", [(1, 64), (3, 64), (5, 128), (32, 64), (48, 64), (64, 64), (96, 128), (127, 64), (128, 64), (160, 64)])
def test_many_rows_of_every_group(G, D):
    """Slots of 128 / G rows: full ones, ragged ones, output boxes and single rows."""
    check([300, 65, 128], [200, 385, 64], 2 * G, 2, D, True, seed=G, num_sms=4)      # two slots an item
    check([130 // G + 70 // min(G, 70), 1], [130, 7], 2 * G, 2, D, False, seed=G, num_sms=1)     # one


def test_large_scores_raise_the_maximum():
    """Scores that pass the first tile's maximum by far; tolerances grow with them (2^-24 (D + 4) of |s| <= 2000: 2^-7)."""
    for qo, sms in (([1, 70], 0), ([5, 200], 3), ([30, 150], 2)):
        q, k, v, s, start, rows = inputs(qo, [900, 1000], 8, 2, 64, True, seed=3)
        k[start[0] + 700] *= 40
        k[start[1] + 999] *= 40
        q = q * 8
        plan = binding().CrossPlan([0, qo[0], sum(qo)], start, [900, 1000], rows, 8, 2, 64, num_sms=sms)
        out, lse = plan.attend(q, k, v, s, lse=torch.empty(sum(qo), 8, device="cuda"))
        want, mag, want_lse = plain(q, k, v, s, qo, start, [900, 1000], 0.125)
        assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -7 + 2.0 ** -6) * mag).all())
        assert bool(((lse.double() - want_lse).abs() <= 2.0 ** -6).all())


def test_infinite_and_nan_states():
    """A NaN in one KV head's keys or values reaches that head's rows of that sequence, and no others."""
    qo, kv = [3, 70, 2], [100, 3000, 40]                     # (the second's keys are split)
    plan, (q, k, v, s), clean, _ = check(qo, kv, 8, 4, 64, False, padded=False, fused=False, seed=5, num_sms=40)
    assert plan.info()["num_prefill_items"] > 4
    k[100 + 250, 1, 7], v[5, 2, 3], v[3099, 0, :] = float("nan"), float("nan"), float("inf")
    out, _ = plan.attend(q, k, v, s)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[3:73, 2:4] = True
    bad[0:3, 4:6, 3] = True
    bad[3:73, 0:2] = True
    assert bool((~torch.isfinite(out[bad])).all()) and torch.equal(out[~bad], clean[~bad])


def test_all_scores_at_minus_infinity():
    """Keys of -inf against positive queries leave nothing to see: as without keys."""
    for rows, sms in ((2, 0), (80, 0), (80, 1)):
        q = torch.ones(rows, 4, 64, dtype=torch.bfloat16, device="cuda")
        k = torch.full((50, 2, 64), -float("inf"), dtype=torch.bfloat16, device="cuda")
        v = torch.ones_like(k)
        plan = binding().CrossPlan([0, rows], [0], [50], 50, 4, 2, 64, num_sms=sms)
        assert (plan.info()["num_prefill_items"] > 0) == (sms == 1)
        out, lse = plan.attend(q, k, v, lse=torch.empty(rows, 4, device="cuda"))
        assert not out.any() and bool((lse == -float("inf")).all())
        sinks = torch.tensor([1.0, -2.0, 0.0, 30.0], device="cuda")
        out, lse = plan.attend(q, k, v, sinks, lse=lse)
        assert not out.any() and torch.allclose(lse, sinks.expand(rows, -1), atol=1e-6, rtol=1e-6)


def test_sequences_that_share_states():
    """Beams as sequences of their own over the same rows, or as rows of one sequence."""
    q, k, v, s, _, rows = inputs([12], [333], 8, 2, 64, True, padded=False, seed=6)
    one = binding().CrossPlan([0, 12], [0], [333], rows, 8, 2, 64).attend(q, k, v, s)[0]
    apart = binding().CrossPlan(range(13), [0] * 12, [333] * 12, rows, 8, 2, 64).attend(q, k, v, s)[0]
    assert float((one.float() - apart.float()).abs().max()) <= 2.0 ** -6 * float(v.float().abs().max())
    want, mag, _ = plain(q, k, v, s, [12], [0], [333], 0.125)
    for out in (one, apart):
        assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -6 * mag).all())


def test_no_states_at_all():
    q = torch.randn(70, 4, 64, device="cuda").to(torch.bfloat16)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    plan = binding().CrossPlan([0, 1, 70], [0, 0], [0, 0], 0, 4, 2, 64)
    out, lse = plan.attend(q, k, k, torch.arange(4.0, device="cuda"), lse=torch.empty(70, 4, device="cuda"))
    assert not out.any() and torch.allclose(lse, torch.arange(4.0, device="cuda").expand(70, -1), atol=1e-6)
    none = binding().CrossPlan([0], [], [], 0, 4, 2, 64)
    assert none.attend(q[:0], k, k)[0].shape == (0, 4, 64)


def test_other_tensors_strides_and_streams_through_one_plan():
    qo, kv = [1, 90, 3], [50, 333, 1000]
    plan, (q, k, v, s), out, lse = check(qo, kv, 16, 4, 64, True, seed=8, num_sms=8)
    assert plan.info()["num_prefill_items"]
    k2, v2 = torch.zeros(len(k), 7, 64, dtype=torch.bfloat16, device="cuda"), v.contiguous()
    k2[:, 2:6] = k
    assert torch.equal(plan.attend(q, k2[:, 2:6], v2, s)[0], out)
    assert torch.equal(plan.attend(q, k, v, s)[0], out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = plan.attend(q.clone(), k, v, s, stream=side)
    side.synchronize()
    assert torch.equal(other, out)


def test_outputs_that_start_in_the_middle_of_a_sector():
    qo, kv = [3, 90, 40], [50, 333, 5000]
    plan, (q, k, v, s), out, lse = check(qo, kv, 16, 4, 64, True, seed=10, num_sms=8)
    assert plan.info()["num_prefill_items"]
    buf = torch.zeros(out.numel() + 16, dtype=torch.bfloat16, device="cuda")
    mine = buf[8:8 + out.numel()].view(out.shape)
    assert mine.data_ptr() % 32 == 16
    plan.attend(q, k, v, s, mine)
    assert torch.equal(mine, out) and not buf[:8].any() and not buf[-8:].any()


def test_captured_and_replayed():
    qo, kv = [1, 5, 200, 2], [70, 9000, 300, 0]
    plan, (q, k, v, s), out, lse = check(qo, kv, 16, 4, 64, True, seed=9, num_sms=8)   # all kernels
    info = plan.info()
    assert info["num_prefill_items"] and info["num_decode_partials"]
    graph = torch.cuda.CUDAGraph()
    plan.attend(q, k, v, s, out, lse)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.attend(q, k, v, s, out, lse)
    for step in range(3):
        q.copy_(torch.randn(q.shape, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        want, want_lse = plan.attend(q, k, v, s, lse=torch.empty_like(lse))
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert plan.device_error() == 0


def test_the_binding_refuses():
    q, k, v, s, start, rows = inputs([3], [20], 8, 2, 64, True, padded=False)
    plan = binding().CrossPlan([0, 3], [0], [20], rows, 8, 2, 64)
    for bad in (dict(q=q.float()), dict(q=q[:2]), dict(k=k[:19]), dict(k=k.cpu()), dict(v=v.transpose(0, 1)),
                dict(v=v[:, :1].expand(-1, 2, -1)), dict(sinks=s[:4]), dict(out=q.float()), dict(lse=s),
                dict(k=torch.as_strided(k, (20, 2, 64), (64, 64, 1)))):
        with pytest.raises((TypeError, ValueError)):
            plan.attend(**{**dict(q=q, k=k, v=v, sinks=s), **bad})
