"""Plain fp64 forms of the compressed-cache operators, for the tests (numpy;
nothing here is used by the library).

The 4-bit pool is uint8 [num_pages, 2, Hkv, P / 16, 9 D]: per 16 tokens, 16
rows of D / 2 code bytes, then 16 rows of D / 16 scale bytes.
"""
import numpy as np

from paged_kv_attention_sink_gb300 import synthetic as syn

CODES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
SCALES = np.array([m / 512 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
SCALES[127] = np.nan
SCALES = np.concatenate([SCALES, -SCALES])


def pool_shape(num_pages, Hkv, P, D):
    return (num_pages, 2, Hkv, P // 16, 9 * D)


def values(pool, D):
    """fp64 [num_pages, 2, Hkv, P, D] of a 4-bit pool, without the pool's scale."""
    codes = pool[..., :8 * D].reshape(*pool.shape[:-1], 16, D // 2)
    scales = pool[..., 8 * D:].reshape(*pool.shape[:-1], 16, D // 16)
    v = CODES[np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D)]
    v = v * np.repeat(SCALES[scales], 16, axis=-1)
    return v.reshape(*pool.shape[:-2], pool.shape[-2] * 16, D)


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0 (ascending grid), a tie to the
    even index, saturating."""
    mid = (grid[1:] + grid[:-1]) / 2                    # exact: few significant bits
    i = np.searchsorted(mid, x, side="left")            # mids strictly below x
    on = (i < len(mid)) & (x == mid[np.minimum(i, len(mid) - 1)])
    return np.where(on & (i % 2 == 1), i + 1, i)


def quantise(bits, pool_scale):
    """bf16 bits [..., D] -> (code bytes [..., D / 2], scale bytes [..., D / 16])."""
    x = syn.bf16_to_float(bits).astype(np.float64) / pool_scale
    g = x.reshape(*x.shape[:-1], -1, 16)
    bad = np.isnan(g).any(-1)
    with np.errstate(invalid="ignore"):
        amax = np.abs(np.where(bad[..., None], 0, g)).max(-1)
        # amax / 6 against the borders, exactly: amax against 6 * border.
        s = nearest(amax, SCALES[:127] * 6)
        f = SCALES[s][..., None]
        # |x| against border * scale (exact); a zero scale takes code 0.
        a = np.abs(g)
        mid = (CODES[1:8] + CODES[:7]) / 2
        code = np.zeros(g.shape, dtype=np.int64)
        for k, m in enumerate(mid):
            code += (a > m * f) if k % 2 == 0 else (a >= m * f)
        code = np.where(f > 0, code, 0) + 8 * np.signbit(g)
    code = code.reshape(x.shape).astype(np.uint8)
    s = np.where(bad, 127, s).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def put_rows(pool, D, page, half, row, bits, pool_scale):
    """Quantise bf16 rows [Hkv, D] into token `row` of a page (in place)."""
    codes, scales = quantise(bits, pool_scale)
    sub, t = row // 16, row % 16
    pool[page, half, :, sub, t * (D // 2):(t + 1) * (D // 2)] = codes
    pool[page, half, :, sub, 8 * D + t * (D // 16):8 * D + (t + 1) * (D // 16)] = scales


def random_pool(rng, num_pages, Hkv, P, D, spread=1.0):
    """Random codes, scales around 0.3 (log-normal)."""
    pool = rng.integers(0, 256, size=pool_shape(num_pages, Hkv, P, D), dtype=np.uint8)
    s = np.exp2(spread * rng.standard_normal(pool[..., 8 * D:].shape) - 2)
    pool[..., 8 * D:] = nearest(s, SCALES[:127]).astype(np.uint8)
    return pool


def poison_unused(pool, batch):
    """NaN scales wherever no request's token lies: a stray read shows."""
    D, P = batch.head_dim, batch.page_size
    used = np.zeros((batch.num_pages, P), dtype=bool)
    for b in range(batch.batch_size):
        t = np.arange(batch.kv_lens[b])
        used[batch.page_table[batch.kv_indptr[b] + t // P], t % P] = True
    page, row = np.nonzero(~used)
    for k in range(D // 16):
        pool[page, :, :, row // 16, 8 * D + (row % 16) * (D // 16) + k] = 0x7F


def gather(batch, pool_values, b, half):
    """fp64 [Hkv, kv_len, D] of request b."""
    pages = batch.page_table[batch.kv_indptr[b]:batch.kv_indptr[b + 1]]
    x = pool_values[pages, half].transpose(1, 0, 2, 3)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :batch.kv_lens[b]]


def attention(batch, pool_values):
    """(out, lse, sum_j p_j |v_j|) of every query row, fp64."""
    Hq, Hkv, D = batch.num_qo_heads, batch.num_kv_heads, batch.head_dim
    G = Hq // Hkv
    out = np.zeros((batch.total_rows, Hq, D))
    mag = np.zeros_like(out)
    lse = np.zeros((batch.total_rows, Hq))
    q = syn.bf16_to_float(batch.q).astype(np.float64)
    for b in range(batch.batch_size):
        k, v = gather(batch, pool_values, b, 0), gather(batch, pool_values, b, 1)
        n, m = int(batch.kv_lens[b]), int(batch.qo_lens[b])
        for i in range(m):
            r = batch.qo_indptr[b] + i
            seen = n - m + i + 1 if batch.causal else n
            for h in range(Hq):
                s = k[h // G, :seen] @ q[r, h] * batch.sm_scale
                top = max(s.max(), -np.inf if batch.sinks is None else batch.sinks[h])
                e = np.exp(s - top)
                tot = e.sum() + (0 if batch.sinks is None else np.exp(np.float64(batch.sinks[h]) - top))
                out[r, h], mag[r, h] = e @ v[h // G, :seen] / tot, e @ np.abs(v[h // G, :seen]) / tot
                lse[r, h] = top + np.log(tot)
    return out, lse, mag


def value_sums(batch, pool_values):
    """sum_j |v_j| over each query row's request and head: [rows, Hq, D]."""
    G = batch.num_qo_heads // batch.num_kv_heads
    per = [np.abs(gather(batch, pool_values, b, 1)).sum(1) for b in range(batch.batch_size)]   # [Hkv, D]
    return np.repeat(np.stack([per[b] for b in np.repeat(np.arange(batch.batch_size), batch.qo_lens)]), G, axis=1)


def key_weights(batch, pool_values, lse, prev, decay, window):
    """(weights, bound on an fp32 evaluation's error) as pools [num_pages, Hkv, P];
    slots that no token takes are NaN."""
    Hq, Hkv, P, D = batch.num_qo_heads, batch.num_kv_heads, batch.page_size, batch.head_dim
    G, u = Hq // Hkv, 2.0 ** -24
    w = np.full((batch.num_pages, Hkv, P), np.nan)
    tol = np.zeros_like(w)
    q = syn.bf16_to_float(batch.q).astype(np.float64)
    for b in range(batch.batch_size):
        n, m = int(batch.kv_lens[b]), int(batch.qo_lens[b])
        if m == 0:
            continue
        k = gather(batch, pool_values, b, 0)
        t = np.arange(n)
        page, row = batch.page_table[batch.kv_indptr[b] + t // P], t % P
        for g in range(Hkv):
            acc, err = np.zeros(n), np.zeros(n)
            if decay:
                old = t < n - m
                acc[old] = decay * prev[page[old], g, row[old]].astype(np.float64)
            terms = 0
            for i in range(max(0, m - window) if window else 0, m):
                seen = n - m + i + 1 if batch.causal else n
                r = batch.qo_indptr[b] + i
                for h in range(g * G, (g + 1) * G):
                    s = k[g, :seen] @ q[r, h] * batch.sm_scale
                    size = np.abs(k[g, :seen]) @ np.abs(q[r, h]) * batch.sm_scale
                    p = np.exp(s - np.float64(lse[r, h]))
                    acc[:seen] += p
                    # exponent: D products summed, scaled, lse subtracted in fp32 (log2 units); ex2: 2^-22.
                    err[:seen] += p * (2.0 ** -22 + u * ((D + 4) * size + 3 * abs(float(lse[r, h]))))
                    terms += 1
            w[page, g, row] = acc
            tol[page, g, row] = err + acc * u * (terms + 8)
    return w, tol


def evict(weights, kv_len, budget, recent):
    """Kept indices (ascending) of one request and head, from its weights [kv_len]."""
    new = max(0, kv_len - recent)
    keep = min(kv_len, budget)
    key = np.where(np.isnan(weights[:new]), -np.inf, weights[:new]) + 0.0
    nan = np.isnan(weights[:new])
    order = np.lexsort((np.arange(new), -key, nan))      # NaN last, then by falling weight, then by index
    return np.sort(np.concatenate([order[:keep - (kv_len - new)], np.arange(new, kv_len)]))
