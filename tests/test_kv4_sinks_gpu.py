"""4-bit decode beside sinks that outweigh every key, and at the ends of a
sink's range.

A sink changes a row's normalisation alone, so the output keeps its relative
accuracy however large the sink is.  Tolerance as in the decode's other tests,
with P's f16 rounding below its normal range, 2^-32 of the largest weight that a
key has (not of the sink's) per key, and 2^-14 for the exponents of up to 2^7
that the parts and the sink are weighed with (fp32: 2^-24 of 2^7 each, a few
of them)."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from helpers import make_plan
from test_kv4_gpu import batch_of, binding, dev, dev_bf16

pytestmark = pytest.mark.gpu


def run(batch, pool, sinks, **kw):
    plan = make_plan(batch, dev(batch.page_table), **kw)
    lse = torch.empty(batch.total_rows, batch.num_qo_heads, device="cuda")
    out, _ = plan.decode_kv4(dev_bf16(batch.q), dev(pool), None if sinks is None else dev(sinks), lse=lse)
    assert plan.device_error() == 0
    return plan, out, lse


@pytest.mark.parametrize("sink", [12.0, 20.0, 30.0, 45.0])
@pytest.mark.parametrize("D,G,P", [(64, 4, 16), (128, 8, 64), (64, 12, 32), (128, 16, 16)])
def test_sinks_above_every_key(D, G, P, sink):
    kv = [1, 33, 64, 300, 5000]
    batch = batch_of([1] * len(kv), kv, G, 1, D, P, seed=G + D)
    pool = ref.random_pool(np.random.default_rng(P), batch.num_pages, 1, P, D)
    ref.poison_unused(pool, batch)
    batch.sinks = (sink + np.random.default_rng(1).standard_normal(G)).astype(np.float32)
    batch.sinks[0] = 0.5                                         # a head without a large sink beside them
    plan, out, lse = run(batch, pool, batch.sinks)
    assert plan.info()["num_decode_groups_split"] > 0
    vals = ref.values(pool, D)
    want, want_lse, mag = ref.attention(batch, vals)
    q = ref.syn.bf16_to_float(batch.q).astype(np.float64)
    top = np.stack([(ref.gather(batch, vals, b, 0)[0] @ q[b].T * batch.sm_scale).max(0) for b in range(len(kv))])
    heaviest = np.exp(top - want_lse)[..., None]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -14) * mag + \
        2.0 ** -32 * heaviest * ref.value_sums(batch, vals) + 1e-36
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -12 + 2.0 ** -22 * np.abs(want_lse))


@pytest.mark.parametrize("num_sms", [0, 1])
def test_sinks_without_end(num_sms):
    """A sink of minus infinity is no sink; one of infinity (exp(inf - inf)) or NaN
    spoils its own head alone."""
    batch = batch_of([1, 1], [900, 40], 4, 1, 64, 16, seed=5)
    pool = ref.random_pool(np.random.default_rng(2), batch.num_pages, 1, 16, 64)
    sinks = np.array([np.inf, -np.inf, np.nan, 1.0], dtype=np.float32)
    _, out, lse = run(batch, pool, sinks, num_sms=num_sms)
    _, plain, plain_lse = run(batch, pool, np.array([0.0, -np.inf, 0.0, 1.0], dtype=np.float32), num_sms=num_sms)
    _, none, none_lse = run(batch, pool, None, num_sms=num_sms)
    assert torch.all(torch.isnan(out[:, [0, 2]])) and torch.all(torch.isnan(lse[:, [0, 2]]))
    assert torch.equal(out[:, 1], none[:, 1]) and torch.equal(lse[:, 1], none_lse[:, 1])
    assert torch.equal(out[:, 3], plain[:, 3]) and torch.equal(lse[:, 3], plain_lse[:, 3])


def test_scores_of_minus_infinity():
    """A query whose products with every key are minus infinity: with a sink the
    output is 0 and the lse the sink, as in the formula; other heads are as
    without it."""
    batch = batch_of([1, 1], [700, 20], 4, 1, 64, 16, seed=6)
    pool = ref.random_pool(np.random.default_rng(3), batch.num_pages, 1, 16, 64)
    pool[:, 0, :, :, :8 * 64] = pool[:, 0, :, :, :8 * 64] & 0x77 | 0x11      # K positive, no zeros
    plain = batch.q.copy()
    batch.q[:, 1] = 0
    batch.q[:, 1, :1] = 0xFF80                                               # -inf in one dim
    batch.q[:, 1, 1:] = 0xBF80                                               # -1 in the others
    batch.sinks = np.array([0.5, -3.0, 1.0, 0.0], dtype=np.float32)
    _, out, lse = run(batch, pool, batch.sinks)
    assert torch.all(out[:, 1] == 0)
    assert torch.all((lse[:, 1] + 3.0).abs() <= 2.0 ** -20)
    batch.q = plain
    _, want, want_lse = run(batch, pool, batch.sinks)
    for h in (0, 2, 3):
        assert torch.equal(out[:, h], want[:, h]) and torch.equal(lse[:, h], want_lse[:, h])


def test_misaligned_sinks_and_lse_are_refused():
    import ctypes
    batch = batch_of([1, 1], [40, 20], 4, 1, 64, 16, seed=7)
    pool = dev(ref.random_pool(np.random.default_rng(1), batch.num_pages, 1, 16, 64))
    plan, q = make_plan(batch, dev(batch.page_table)), dev_bf16(batch.q)
    out, f = torch.full_like(q, 3.0), torch.zeros(16, device="cuda")
    at = lambda t, off=0: ctypes.c_void_p(t.data_ptr() + off)
    call = binding().load_library().attn_decode_kv4
    stream = torch.cuda.current_stream().cuda_stream
    for sinks, lse in ((at(f, 2), None), (None, at(f, 1)), (at(f, 3), at(f, 2))):
        assert call(plan.handle, at(q), at(pool), 1.0, 1.0, sinks, at(out), lse, stream) == 1
    torch.cuda.synchronize()
    assert torch.all(out == 3.0)
    assert call(plan.handle, at(q), at(pool), 1.0, 1.0, at(f, 4), at(out), at(f, 32), stream) == 0
    assert plan.device_error() == 0 and not torch.any(out == 3.0)
