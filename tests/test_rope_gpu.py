"""Rotary positions on the GPU against the plain 64-bit form.

Tolerance.  The angle in half turns is rounded to fp32 (2^-25 below 1, so pi *
2^-25 < 2^-23 in radians; its fixed-point form adds 2^-31 of a turn at most);
sincospif is good to 2 units in the last place, 2^-23 for values below 1; the
product with scale, the product and the fused multiply-add round by 2^-24 each.
In all below 2^-21 of scale (|x| + |y|) of the pair, and then half a step of
bf16, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import rope_reference as ref
from helpers import make_plan, syn

pytestmark = pytest.mark.gpu


def binding():
    from paged_kv_attention_sink_gb300 import binding
    return binding


def rows_of(rows, heads, D, slack=0, seed=0):
    """bf16 rows that lie `slack` elements further apart than they need to."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(max(rows, 1), heads * D + slack, device="cuda", generator=g).to(torch.bfloat16)
    return x[:rows, :heads * D].unflatten(1, (heads, D))


def check(out, x, cos, sin, inter, scale=1.0, inverse=False):
    want, mag = ref.turned(x.double().cpu().numpy(), cos, sin, inter, scale, inverse)
    err = np.abs(out.double().cpu().numpy() - want)
    tol = 2.0 ** -21 * mag + 2.0 ** -8 * np.abs(want) + 1e-38
    same = mag == 0                                        # dims that do not turn are copied
    assert np.array_equal(out.double().cpu().numpy()[same], want[same])
    assert np.all(err <= tol), float((err / tol).max())


CASES = [  # rows, Hq, Hkv, D, rot, axes, interleaved, inverse, scale, slack
    (1, 1, 1, 64, 64, 1, False, False, 1.0, 0),
    (1, 8, 2, 128, 128, 1, False, False, 1.0, 64),
    (3, 5, 1, 64, 16, 2, False, True, 1.0, 8),
    (7, 12, 3, 128, 112, 3, False, False, 1.25, 24),
    (65, 16, 16, 64, 48, 4, True, False, 0.5, 0),
    (130, 64, 8, 64, 64, 1, True, True, 1.0, 136),
    (1217, 4, 4, 128, 96, 8, False, True, 1.0, 8),
    (1221, 3, 1, 128, 16, 3, True, False, 2.0, 0),
    (6001, 1, 1, 64, 64, 2, False, False, 1.0, 0),          # few heads: many rows to a CTA
    (5000, 2, 1, 128, 128, 2, True, True, 1.0, 8),
    (1500, 64, 4, 128, 128, 3, False, False, 1.0, 0),
]


@pytest.mark.parametrize("rows,Hq,Hkv,D,rot,axes,inter,inverse,scale,slack", CASES)
def test_against_the_plain_form(rows, Hq, Hkv, D, rot, axes, inter, inverse, scale, slack):
    rng = np.random.default_rng(rows)
    freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    axis = rng.integers(0, axes, rot // 2)
    axis[-1] = axes - 1
    pos = rng.integers(0, 600, (axes, rows)).astype(np.int32)
    rope = binding().Rope(freq, axis=axis, interleaved=inter, scale=scale)
    assert rope.n_axes == axes and rope.rot_dim == rot
    q, k = rows_of(rows, Hq, D, slack, 1), rows_of(rows, Hkv, D, slack, 2)
    qo, ko = rope.apply(torch.from_numpy(pos).cuda(), q, k, inverse=inverse)
    cos, sin = ref.cos_sin(pos, freq, axis)
    check(qo, q, cos, sin, inter, scale, inverse)
    check(ko, k, cos, sin, inter, scale, inverse)
    # One tensor at a time, strided outputs whose gaps stay, and in place.
    wide = torch.full((rows, Hq * D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = rope.apply(torch.from_numpy(pos).cuda(), q, q_out=wide[:, :Hq * D].unflatten(1, (Hq, D)), inverse=inverse)
    assert torch.equal(out, qo) and bool((wide[:, Hq * D:] == 7.0).all())
    again = q.clone() if slack == 0 else q
    rope.apply(torch.from_numpy(pos).cuda(), again, k, q_out=again, k_out=k, inverse=inverse)
    assert torch.equal(again, qo) and torch.equal(k, ko)


def test_far_and_negative_positions():
    rng = np.random.default_rng(5)
    freq = np.concatenate([[1.0, 0.5, 2.0 ** -20, 1e-4, 0.9999999, 3.14159274, 1000.5, 2.0 ** 19, -0.3, 0.0],
                           rng.uniform(0, 1, 22)]).astype(np.float32)
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -(2 ** 31), 10 ** 9 + 7, -123456789, 2 ** 24 + 1]], dtype=np.int32)
    rope = binding().Rope(freq)
    q = rows_of(8, 3, 64, 0, 3)
    out = rope.apply(torch.from_numpy(pos[0]).cuda(), q)
    cos, sin = ref.cos_sin(pos, freq, [0] * 32)
    check(out, q, cos, sin, False)


def test_rows_further_apart_than_32_bits():
    buf = torch.zeros((3 << 30) + 4096, dtype=torch.bfloat16, device="cuda")        # 6.4 GB
    q = torch.as_strided(buf, (4, 3, 64), (1 << 30, 64, 1))
    q.copy_(rows_of(4, 3, 64, 0, 8))
    rope = binding().Rope((0.9 ** np.arange(32)).astype(np.float32))
    pos = torch.tensor([3, 1, 4, 100], dtype=torch.int32, device="cuda")
    want = rope.apply(pos, q.contiguous())
    assert torch.equal(rope.apply(pos, q), want)
    rope.apply(pos, q, q_out=q)
    assert torch.equal(q, want)


def test_it_is_its_gradient_transposed():
    """out = R q, so the gradient of sum(w out) by q is R^T w: against autograd and differences of the 64-bit form."""
    freq = (100.0 ** (-np.arange(24) / 24)).astype(np.float32)
    axis = [p % 3 for p in range(24)]
    pos = np.random.default_rng(1).integers(0, 90, (3, 5)).astype(np.int32)
    cos, sin = ref.cos_sin(pos, freq, axis)
    w = rows_of(5, 2, 64, 0, 9)
    got = binding().Rope(freq, axis=axis, interleaved=True, scale=1.5).apply(torch.from_numpy(pos).cuda(), w, inverse=True)
    c, s = torch.from_numpy(cos)[:, None], torch.from_numpy(sin)[:, None]

    def forward(x):
        a, b = x[..., 0:48:2], x[..., 1:48:2]
        return torch.cat((1.5 * torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2), x[..., 48:]), -1)

    x = torch.randn(5, 2, 64, dtype=torch.float64, requires_grad=True)
    wd = w.double().cpu()
    (forward(x) * wd).sum().backward()
    tol = 2.0 ** -8 * x.grad.abs() + 2.0 ** -21 * 1.5 * 2 * wd.abs().amax(-1, keepdim=True)
    assert bool(((got.double().cpu() - x.grad).abs() <= tol).all())
    for d in (0, 13, 47, 60):                              # the form is linear: a difference of any width is exact
        e = torch.zeros_like(x)
        e[2, 1, d] = 1.0
        diff = ((forward(x.detach() + e) - forward(x.detach())) * wd).sum()
        assert abs(float(diff - x.grad[2, 1, d])) < 1e-12 * (1 + float(wd.abs().sum()))


def test_infinities_and_nan_stay_in_their_pair():
    q = rows_of(2, 2, 64, 0, 4)
    clean = q.clone()
    q[0, 1, 3] = float("nan")
    q[1, 0, 40] = float("inf")
    rope = binding().Rope((0.9 ** np.arange(32)).astype(np.float32))
    pos = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    out, want = rope.apply(pos, q), rope.apply(pos, clean)
    bad = torch.zeros(2, 2, 64, dtype=torch.bool, device="cuda")
    bad[0, 1, [3, 35]] = True
    bad[1, 0, [8, 40]] = True
    assert bool((~torch.isfinite(out[bad])).all()) and torch.equal(out[~bad], want[~bad])


def batch_of(qo, kv, Hq, Hkv, D, P, seed=0):
    return syn.make_batch("rope", qo, kv, Hq, Hkv, D, P, seed=seed, fill_pool=False)


@pytest.mark.parametrize("qo,kv,Hq,Hkv,D,P,inter", [
    ([1], [1], 1, 1, 64, 16, False), ([1] * 9, [1, 16, 17, 300, 31, 32, 33, 64, 5], 64, 8, 64, 16, False),
    ([5, 0, 1, 40], [70, 3, 9, 40], 12, 3, 128, 32, True), ([700, 1, 611], [900, 65, 611], 10, 2, 128, 128, False)])
def test_append_is_apply_and_append(qo, kv, Hq, Hkv, D, P, inter):
    batch = batch_of(qo, kv, Hq, Hkv, D, P, seed=len(qo))
    rows = batch.total_rows
    pt = torch.from_numpy(batch.page_table).cuda()
    plan = make_plan(batch, pt)
    rope = binding().Rope((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32), axis=[p % 2 for p in range(D // 2)],
                          interleaved=inter)
    fused = rows_of(rows, Hq + 2 * Hkv, D, 0, 7)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    pos = torch.randint(0, 9000, (2, rows), device="cuda", dtype=torch.int32)
    pool = torch.randint(-30000, 30000, (batch.num_pages, 2, Hkv, P, D), dtype=torch.int16, device="cuda").view(torch.bfloat16)
    want = pool.clone()
    qo_want, k_want = rope.apply(pos, q, k)
    plan.append_kv(k_want, v.contiguous(), want)
    got = plan.append_kv_rope(rope, pos, q, k, v, pool)
    assert torch.equal(got, qo_want)
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    assert plan.device_error() == 0
    # q in place, on another stream
    side, mine = torch.cuda.Stream(), q.contiguous()
    side.wait_stream(torch.cuda.current_stream())
    plan.append_kv_rope(rope, pos, mine, k, v, pool, q_out=mine, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(mine, qo_want) and torch.equal(pool.view(torch.int16), want.view(torch.int16))


def test_a_page_outside_the_pool_is_skipped_and_flagged():
    batch = batch_of([1, 1, 3], [20, 33, 18], 4, 2, 64, 16)
    table = batch.page_table.copy()
    table[batch.kv_indptr[1] + 2] = batch.num_pages
    table[batch.kv_indptr[2]] = -5
    plan = make_plan(batch, torch.from_numpy(table).cuda())
    rope = binding().Rope(np.ones(32, np.float32))
    q, k, v = rows_of(5, 4, 64), rows_of(5, 2, 64, 0, 1), rows_of(5, 2, 64, 0, 2)
    pos = torch.arange(5, device="cuda", dtype=torch.int32)
    pool = torch.zeros(batch.num_pages, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q_out = plan.append_kv_rope(rope, pos, q, k, v, pool)
    assert plan.device_error() == 1
    q_want, k_want = rope.apply(pos, q, k)
    assert torch.equal(q_out, q_want)
    want = torch.zeros_like(pool)
    for row, (slot, at) in {0: (batch.kv_indptr[0] + 1, 3), 3: (batch.kv_indptr[2] + 1, 0), 4: (batch.kv_indptr[2] + 1, 1)}.items():
        want[table[slot], 0, :, at], want[table[slot], 1, :, at] = k_want[row], v[row]
    assert torch.equal(pool, want)


def test_captured_and_replayed_with_other_positions():
    batch = batch_of([1] * 6, [40, 1, 17, 16, 90, 33], 8, 2, 64, 16)
    plan = make_plan(batch, torch.from_numpy(batch.page_table).cuda())
    rope = binding().Rope((0.8 ** np.arange(32)).astype(np.float32))
    q, k, v = rows_of(6, 8, 64), rows_of(6, 2, 64, 0, 1), rows_of(6, 2, 64, 0, 2)
    pos = torch.arange(6, device="cuda", dtype=torch.int32)
    pool = torch.zeros(batch.num_pages, 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty_like(q)
    plan.append_kv_rope(rope, pos, q, k, v, pool, q_out=q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.append_kv_rope(rope, pos, q, k, v, pool, q_out=q_out)
        turned = rope.apply(pos, q_out, inverse=True)
    for step in range(3):
        pos.add_(1000)
        q.copy_(rows_of(6, 8, 64, 0, 20 + step))
        graph.replay()
        torch.cuda.synchronize()
        want = rope.apply(pos, q)
        assert torch.equal(q_out, want) and torch.equal(turned, rope.apply(pos, want, inverse=True))


def test_the_binding_refuses():
    rope = binding().Rope(np.ones(32, np.float32), axis=[0] * 16 + [1] * 16)
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    q = rows_of(4, 2, 64)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(positions=pos[0]), dict(q=q.float()),
                dict(q=q.transpose(0, 1)), dict(q=rows_of(4, 2, 64, 4)), dict(q=torch.as_strided(q, (4, 2, 64), (64, 64, 1))),
                dict(k=q[:3]), dict(k=q.cpu()), dict(k_out=q), dict(q_out=q[:, :1])):
        with pytest.raises((TypeError, ValueError)):
            rope.apply(**{**dict(positions=pos, q=q), **bad})
    with pytest.raises(binding().AttnError):
        rope.apply(pos, torch.zeros(4, 2, 32, dtype=torch.bfloat16, device="cuda"))
    assert rope.apply(pos[:, :0].contiguous(), q[:0]).shape == (0, 2, 64)
