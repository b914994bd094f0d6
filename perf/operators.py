"""Cases of the compressed KV cache's operators, for measuring them.

A cache is kept small in two ways: its rows are held in 4 bits, and the keys
that attention hardly looks at are dropped.  The operators:

  store    write a step's K/V rows into the 4-bit pages, then read pages back
           in bf16 (what a chunked prefill over such a cache reads)
  decode4  sink attention of one query token per request over the 4-bit pages
  weights  the attention weight each cached key receives from the step's
           queries, added to what it had received before
  evict    keep each KV head's most attended keys and the newest ones, moved
           into the request's new pages

``run`` computes an operator in elementary torch operations, or, where ``own``
is set, through the library's entry points on the same inputs.

The 4-bit page: uint8 [num_pages][2][Hkv][P / 16][16 * D / 2 + 16 * D / 16]; a
(page, K/V, KV head) block holds its tokens in sixteens, each 16 rows of D / 2
bytes (dim 2i in the low nibble of byte i, dim 2i + 1 in the high one; sign and
e2m1 magnitude), then 16 rows of D / 16 e4m3 scales, one per 16 dims.  A value
is e2m1 * e4m3 * k_scale (v_scale).
"""
import math
import random

import torch

own = False

GROUP = 16                                           # dims that share a scale
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1


# ------------------------------------------------------------------- cases

def listed():
    gptoss = dict(Hq=64, Hkv=8, D=64, P=16)
    qwen = dict(Hq=64, Hkv=4, D=128, P=64)
    step = dict(batch=64, kv_lo=1024, kv_hi=8192, lens=0)
    return [
        # The append of one decode step, and each request's page in progress read back.
        dict(name="store_step", op="store", **step, qo=1, pages="last", v_scale=1.0, **gptoss),
        # Chunked prefill: 2048 new rows per request; the whole prefix is read back for attention.
        dict(name="store_chunks", op="store", batch=4, kv_lo=2048, kv_hi=10240, lens=1, qo=2048, pages="all",
             v_scale=0.0625, **gptoss),
        # Long prompts of odd lengths, stored and read back whole.
        dict(name="store_prompts", op="store", batch=8, kv_lo=6000, kv_hi=8192, lens=2, qo=0, pages="all",
             v_scale=1.0, Hq=64, Hkv=8, D=128, P=64),
        # The smallest decode: two short requests, where latency is all.
        dict(name="decode4_tiny", op="decode4", batch=2, kv_lo=97, kv_hi=256, lens=0, sinks=True, v_scale=1.0,
             Hq=8, Hkv=2, D=64, P=16),
        # An ordinary serving step.
        dict(name="decode4_step", op="decode4", **step, sinks=True, v_scale=1.0, **gptoss),
        # A large batch of very uneven lengths.
        dict(name="decode4_many", op="decode4", batch=256, kv_lo=512, kv_hi=16384, lens=3, sinks=True,
             v_scale=0.0625, **gptoss),
        # Long contexts, sixteen query heads on each KV head, no sinks.
        dict(name="decode4_long", op="decode4", batch=32, kv_lo=2048, kv_hi=32768, lens=4, sinks=False, v_scale=1.0,
             **qwen),
        # What one decode step adds to every key's weight, over bf16 pages.
        dict(name="weights_step", op="weights", **step, qo=1, window=0, bits=16, decay=1.0, **gptoss),
        # The same over 4-bit pages of long contexts, older steps counting less.
        dict(name="weights_step4", op="weights", batch=32, kv_lo=2048, kv_hi=32768, lens=4, qo=1, window=0, bits=4,
             decay=0.96875, **qwen),
        # A prompt's keys, scored by all of the prompt's queries under the causal mask.
        dict(name="weights_prompts", op="weights", batch=4, kv_lo=512, kv_hi=4096, lens=5, qo=0, window=0, bits=16,
             decay=1.0, **gptoss),
        # Down to 1024 keys per head after a decode step.
        dict(name="evict_step", op="evict", **step, qo=1, budget=1024, recent=128, bits=16, **gptoss),
        # Long contexts in 4 bits down to 4000 keys per head, then read back in bf16.
        dict(name="evict_long4", op="evict", batch=32, kv_lo=2048, kv_hi=32768, lens=4, qo=1, budget=4000, recent=64,
             bits=4, **qwen),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "decode4", "decode4", "weights", "weights", "evict"])
    D = rng.choice([64, 128])
    P = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16])
    kv_hi = _spread(rng, 2, 32768)
    kv_lo = max(1, int(kv_hi * rng.uniform(0.05, 1.0)))
    batch = max(1, min(_spread(rng, 1, 256), (1 << 28) // (kv_hi * Hkv * D)))
    case = dict(op=op, batch=batch, kv_lo=kv_lo, kv_hi=kv_hi, lens=rng.randrange(1 << 20), Hq=Hkv * G, Hkv=Hkv, D=D,
                P=P)
    v_scale = 2.0 ** rng.randint(-6, 2)
    if op == "store":
        case.update(qo=rng.choice([0, 1, _spread(rng, 1, kv_hi)]), pages=rng.choice(["last", "all"]), v_scale=v_scale)
    elif op == "decode4":
        case.update(sinks=rng.random() < 0.7, v_scale=v_scale)
    elif op == "weights":
        qo = rng.choice([0, 1, 1, _spread(rng, 1, kv_hi)])
        rows = kv_hi if qo == 0 else qo
        while case["batch"] * case["Hq"] * rows * case["kv_hi"] > 1 << 31 and case["batch"] > 1:
            case["batch"] = max(1, case["batch"] // 2)
        while case["Hq"] * rows * case["kv_hi"] > 1 << 31:
            case["kv_hi"] = kv_hi = max(2, kv_hi // 2 + 1)
            case["kv_lo"] = max(1, case["kv_lo"] // 2)
            rows = kv_hi if qo == 0 else min(qo, kv_hi)
        case.update(qo=qo, window=rng.choice([0, 0, 32, _spread(rng, 1, 512)]), bits=rng.choice([16, 4]),
                    decay=rng.choice([1.0, 0.96875, 0.0]))
    else:
        budget = _spread(rng, 1, kv_hi)
        case.update(qo=1, budget=budget, recent=rng.randint(0, budget), bits=rng.choice([16, 4]))
    return case


def _kv_lens(case):
    """Lengths of the case's requests, the shortest and the longest allowed among them."""
    rng = random.Random(case["lens"])
    lens = [rng.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["batch"])]
    lens[0] = case["kv_hi"]
    if len(lens) > 1:
        lens[1] = case["kv_lo"]
    return lens


def _qo_lens(case):
    want = case.get("qo", 1)
    return [n if want == 0 else min(want, n) for n in _kv_lens(case)]


def _first_rows(case):
    """Query rows that count: the last `window` of each request (0: all)."""
    w = case.get("window", 0)
    return [max(0, n - w) if w else 0 for n in _qo_lens(case)]


def _csr(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _pages_of(lens, P):
    return [(n + P - 1) // P for n in lens]


def work(case):
    D, Hq, Hkv, P = case["D"], case["Hq"], case["Hkv"], case["P"]
    kv, qo = _kv_lens(case), _qo_lens(case)
    row4 = D // 2 + D // GROUP                       # bytes of a 4-bit row
    tokens, rows = sum(kv), sum(qo)
    if case["op"] == "store":
        pages = case["batch"] if case["pages"] == "last" else sum(_pages_of(kv, P))
        back = 2 * pages * P * Hkv
        return {"bytes": 2 * rows * Hkv * (2 * D + row4) + back * (row4 + 2 * D), "flops": 4 * rows * Hkv * D}
    if case["op"] == "decode4":
        return {"bytes": 2 * tokens * Hkv * row4 + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * tokens}
    if case["op"] == "weights":
        pairs = sum(sum(min(n, n - q + i + 1) for i in range(f, q)) for n, q, f in zip(kv, qo, _first_rows(case)))
        old = sum(n - q for n, q in zip(kv, qo)) if case["decay"] else 0
        used = sum(q - f for q, f in zip(qo, _first_rows(case)))
        return {"bytes": tokens * Hkv * (2 * D if case["bits"] == 16 else row4) + 4 * Hkv * (tokens + old) +
                used * Hq * (2 * D + 4), "flops": 2 * D * Hq * pairs}
    kept = [min(n, case["budget"]) for n in kv]
    row = 2 * D if case["bits"] == 16 else row4
    back = 0 if case["bits"] == 16 else 2 * Hkv * P * sum(_pages_of(kept, P)) * (row4 + 2 * D)
    return {"bytes": 4 * Hkv * tokens + Hkv * sum(kept) * (4 * row + 8) + back, "flops": Hkv * tokens}


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _kv_rows(g, rows, Hkv, D, v_scale):
    """K rows with channels of uneven size, V rows around v_scale; bf16."""
    k = _normal(g, rows, Hkv, D) * torch.exp(0.4 * _normal(g, Hkv, D))
    v = _normal(g, rows, Hkv, D) * v_scale
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _pool4(g, num_pages, Hkv, P, D):
    """A 4-bit pool as bell-shaped rows leave it: codes by their share, and scales within a few octaves of 0.4."""
    n = num_pages * 2 * Hkv * (P // 16)
    codes = (_normal(g, n, 8 * D).abs_() * 3.0).clamp_(max=6.49).to(torch.uint8)
    high = torch.randint(0, 16, (n, 8 * D), device="cuda", generator=g, dtype=torch.uint8)
    scale = torch.exp2(0.7 * _normal(g, n, D) - 1.3).to(torch.float8_e4m3fn).view(torch.uint8)
    both = codes | (high & 8) | ((high ^ (codes >> 1)) << 4)
    return torch.cat([both, scale], dim=1).view(num_pages, 2, Hkv, P // 16, 9 * D)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, Hq, Hkv, P, op = case["D"], case["Hq"], case["Hkv"], case["P"], case["op"]
    kv, qo = _kv_lens(case), _qo_lens(case)
    n_pages = _pages_of(kv, P)
    indptr, qo_indptr = _csr(n_pages), _csr(qo)
    total = indptr[-1]
    num_pages = total + max(1, total // 4)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {
        "case": dict(case), "max_kv": max(kv), "max_qo": max(qo), "num_pages": num_pages,
        "host": dict(qo_indptr=qo_indptr, kv_indptr=indptr, last_page_len=[n - (m - 1) * P for n, m in zip(kv, n_pages)]),
        "kv_len": torch.tensor(kv, device="cuda"), "qo_len": torch.tensor(qo, device="cuda"),
        "indptr": torch.tensor(indptr, device="cuda"), "qo_indptr": torch.tensor(qo_indptr, device="cuda"),
        "page_table": torch.randperm(num_pages, device="cuda", generator=g)[:total].to(torch.int32),
        "k_scale": 1.0, "v_scale": case.get("v_scale", 1.0), "sm_scale": D ** -0.5,
    }
    if op == "store" or op == "decode4" or case.get("bits") == 4:
        s["pool"] = _pool4(g, num_pages, Hkv, P, D)
    else:
        pool = torch.empty(num_pages, 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
        s["pool"] = pool.normal_(generator=g)
    rows = qo_indptr[-1]
    if op == "store":
        s["k_new"], s["v_new"] = _kv_rows(g, rows, Hkv, D, s["v_scale"])
        last = torch.tensor(indptr[1:], device="cuda") - 1
        s["page_ids"] = (s["page_table"][last] if case["pages"] == "last" else s["page_table"]).contiguous()
        s["back"] = torch.zeros(s["page_ids"].numel(), 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
    if op in ("decode4", "weights"):
        s["q"] = _normal(g, rows, Hq, D).to(torch.bfloat16)
        s["sinks"] = _normal(g, Hq) if case.get("sinks") else None
    if op == "decode4":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, Hq, device="cuda")
    if op == "weights":
        # The rows' log-sum-exp, as attention returns it: of n keys with normal scores.
        b = torch.repeat_interleave(torch.arange(len(kv), device="cuda"), s["qo_len"])
        pos = s["kv_len"][b] - s["qo_len"][b] + torch.arange(rows, device="cuda") - s["qo_indptr"][b] + 1
        spread = s["q"].float().square().sum(-1) * (0.5 / D)
        s["lse"] = (pos.float().log()[:, None] + spread.clamp(max=20.0)).contiguous()
        s["prev"] = torch.exp(2.0 * _normal(g, num_pages, Hkv, P) - 3.0)
        s["weights"] = torch.zeros(num_pages, Hkv, P, device="cuda")
    if op == "evict":
        # Heavy-tailed weights; a tenth of the keys never attended to at all, and some equal ones.
        w = torch.exp(2.0 * _normal(g, num_pages, Hkv, P) - 3.0)
        w = torch.where(w > 0.02, w, torch.zeros_like(w))
        s["weights"] = torch.where(w < 0.08, (w * 256).round() / 256, w).contiguous()
        keep = [min(n, case["budget"]) for n in kv]
        out_pages = _csr(_pages_of(keep, P))
        pool_out = out_pages[-1] + 3
        s["keep"] = torch.tensor(keep, device="cuda")
        s["out_indptr"] = torch.tensor(out_pages, device="cuda")
        s["out_table"] = torch.randperm(pool_out, device="cuda", generator=g)[:out_pages[-1]].to(torch.int32)
        s["pool_out"] = torch.zeros(pool_out, *s["pool"].shape[1:], dtype=s["pool"].dtype, device="cuda")
        s["weights_out"] = torch.zeros(pool_out, Hkv, P, device="cuda")
        s["kept"] = torch.empty(len(kv), Hkv, case["budget"], **i32)
        if case["bits"] == 4:
            s["back"] = torch.empty(out_pages[-1], 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _table(device):
    return torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=device)


def _views(pool, D):
    """A pool's code bytes [..., P / 16, 16, D / 2] and scale bytes [..., P / 16, 16, D / 16]."""
    return pool[..., :8 * D].unflatten(-1, (16, D // 2)), pool[..., 8 * D:].unflatten(-1, (16, D // GROUP))


def _unpack(blocks, D):
    """[..., P / 16, 9 * D] bytes -> fp32 [..., P, D], without the pool's scale."""
    rows, scales = _views(blocks, D)
    scales = scales.contiguous().view(torch.float8_e4m3fn).float()
    codes = torch.stack([rows & 15, rows >> 4], dim=-1).flatten(-2)
    return (_table(blocks.device)[codes.int()] * scales.repeat_interleave(GROUP, dim=-1)).flatten(-3, -2)


def _pack(x, scale):
    """bf16 [..., D] -> (bytes [..., D / 2], scale bytes [..., D / 16])."""
    x = x.float().unflatten(-1, (-1, GROUP)) / scale          # a power of two: exact
    s = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f, a = s.float()[..., None], x.abs()
    # The borders between neighbouring magnitudes, times the scale, are exact; a tie goes to the even code.
    code = ((a > 0.25 * f).int() + (a >= 0.75 * f) + (a > 1.25 * f) + (a >= 1.75 * f) + (a > 2.5 * f) + (a >= 3.5 * f) +
            (a > 5.0 * f))
    code = torch.where(f > 0, code, torch.zeros_like(code)) + 8 * (x < 0)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _token_pages(s, t):
    """Page id and row in the page of tokens t [..., n] of each request ([B, n])."""
    P = s["case"]["P"]
    slot = (s["indptr"][:-1, None] + t // P).clamp(max=s["page_table"].numel() - 1)
    return s["page_table"][slot].long(), t % P


def _rows_of(s):
    """Request and position of every query row."""
    rows = torch.arange(s["host"]["qo_indptr"][-1], device="cuda")
    b = torch.searchsorted(s["qo_indptr"], rows, right=True) - 1
    return b, s["kv_len"][b] - s["qo_len"][b] + rows - s["qo_indptr"][b]


def _gather_kv(s, half):
    """K (0) or V (1) of every request, padded: fp32 [B, Hkv, T, D]."""
    P, D = s["case"]["P"], s["case"]["D"]
    n = (s["max_kv"] + P - 1) // P
    pages = _token_pages(s, torch.arange(n, device="cuda")[None] * P)[0]
    x = s["pool"][pages, half]
    x = _unpack(x, D) * (s["v_scale"] if half else s["k_scale"]) if x.dtype == torch.uint8 else x.float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :s["max_kv"]]


def _plain_expand(pool, page_ids, D, k_scale, v_scale):
    f = torch.tensor([k_scale, v_scale], device="cuda")[None, :, None, None, None]
    return (_unpack(pool[page_ids.long()], D) * f).to(torch.bfloat16)


def _plain_store(s):
    P, D = s["case"]["P"], s["case"]["D"]
    b, t = _rows_of(s)
    page, row = s["page_table"][s["indptr"][b] + t // P].long(), t % P
    codes, scales = _views(s["pool"], D)
    kb, ks = _pack(s["k_new"], s["k_scale"])
    vb, vs = _pack(s["v_new"], s["v_scale"])
    codes[page, 0, :, row // 16, row % 16], scales[page, 0, :, row // 16, row % 16] = kb, ks
    codes[page, 1, :, row // 16, row % 16], scales[page, 1, :, row // 16, row % 16] = vb, vs
    return _plain_expand(s["pool"], s["page_ids"], D, s["k_scale"], s["v_scale"])


def _plain_decode4(s):
    c = s["case"]
    k, v = _gather_kv(s, 0), _gather_kv(s, 1)
    q = s["q"].float().unflatten(1, (c["Hkv"], -1))
    x = torch.einsum("bhgd,bhtd->bhgt", q, k) * s["sm_scale"]
    t = torch.arange(s["max_kv"], device="cuda")
    x = x.masked_fill(t >= s["kv_len"][:, None, None, None], float("-inf"))
    v = torch.where((t < s["kv_len"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    m = x.amax(-1, keepdim=True)
    sink = torch.full_like(m, float("-inf")) if s["sinks"] is None else \
        s["sinks"].view(1, c["Hkv"], -1, 1).expand_as(m)
    m = torch.maximum(m, sink)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True) + torch.exp(sink - m)
    out = torch.einsum("bhgt,bhtd->bhgd", e, v) / total
    return out.flatten(1, 2).to(torch.bfloat16), (m + total.log()).flatten(1)


def _plain_weights(s):
    c = s["case"]
    k = _gather_kv(s, 0)
    # Query rows that count, padded to [B, n].
    first = (s["qo_len"] - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(s["qo_len"])
    n = min(s["max_qo"], c["window"]) if c["window"] else s["max_qo"]
    i = first[:, None] + torch.arange(n, device="cuda")
    live = i < s["qo_len"][:, None]
    row = (s["qo_indptr"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (c["Hkv"], -1))                       # [B, n, Hkv, G, D]
    lse = s["lse"][row].unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1)       # [B, Hkv, G, n]
    x = torch.einsum("bnhgd,bhtd->bhgnt", q, k)
    x.mul_(s["sm_scale"]).sub_(lse[..., None]).exp_()
    t = torch.arange(s["max_kv"], device="cuda")
    pos = (s["kv_len"] - s["qo_len"])[:, None] + i
    seen = live[..., None] & (t <= pos[..., None]) & (t < s["kv_len"][:, None, None])
    x.masked_fill_(~seen[:, None, None], 0.0)
    w = x.sum((2, 3))                                                          # [B, Hkv, T]
    page, r = _token_pages(s, t[None].expand(len(w), -1))
    old = (s["kv_len"] - s["qo_len"])[:, None] > t
    if c["decay"]:
        before = s["prev"][page, :, r].transpose(1, 2)
        w = w + torch.where(old[:, None], c["decay"] * before, torch.zeros_like(w))
    here = t < s["kv_len"][:, None]
    s["weights"][page[here], :, r[here]] = w.transpose(1, 2)[here]
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    P, D, Hkv, budget = c["P"], c["D"], c["Hkv"], c["budget"]
    t = torch.arange(s["max_kv"], device="cuda")
    page, r = _token_pages(s, t[None].expand(c["batch"], -1))
    w = s["weights"][page, :, r].transpose(1, 2)                               # [B, Hkv, T]
    n = s["kv_len"][:, None, None]
    key = w.masked_fill(t >= n - c["recent"], float("inf")).masked_fill(t >= n, float("-inf"))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    order = torch.nn.functional.pad(order, (0, max(0, budget - s["max_kv"])))[..., :budget]
    j = torch.arange(budget, device="cuda")
    used = j < s["keep"][:, None]                                              # [B, budget]
    src = torch.where(used[:, None], order, torch.full_like(order, 1 << 30)).sort(-1).values
    s["kept"].copy_(torch.where(used[:, None], src, torch.full_like(src, -1)))
    b, i = used.nonzero(as_tuple=True)
    src = src[b, :, i]                                                         # [kept, Hkv]
    head = torch.arange(Hkv, device="cuda").expand_as(src)
    page, r = s["page_table"][s["indptr"][b][:, None] + src // P].long(), src % P
    page_out = s["out_table"][s["out_indptr"][b] + i // P].long()[:, None].expand_as(src)
    row_out = (i % P)[:, None].expand_as(src)
    s["weights_out"][page_out, head, row_out] = s["weights"][page, head, r]
    if c["bits"] == 16:
        s["pool_out"].transpose(1, 2)[page_out, head, :, row_out] = s["pool"].transpose(1, 2)[page, head, :, r]
        return s["kept"], s["pool_out"], s["weights_out"]
    codes, scales = _views(s["pool"].transpose(1, 2), D)
    codes_out, scales_out = _views(s["pool_out"].transpose(1, 2), D)
    codes_out[page_out, head, :, row_out // 16, row_out % 16] = codes[page, head, :, r // 16, r % 16]
    scales_out[page_out, head, :, row_out // 16, row_out % 16] = scales[page, head, :, r // 16, r % 16]
    back = _plain_expand(s["pool_out"], s["out_table"], D, s["k_scale"], s["v_scale"])
    return s["kept"], back, s["weights_out"]


# ---------------------------------------------------- the library's operators

def _own_plan(s):
    """The step's plan, made once per batch as a serving loop does (every layer uses it)."""
    if "plan" not in s:
        from paged_kv_attention_sink_gb300 import binding
        c, h = s["case"], s["host"]
        s["binding"] = binding
        s["plan"] = binding.Plan(h["qo_indptr"], h["kv_indptr"], s["page_table"], h["last_page_len"], c["Hq"], c["Hkv"],
                                 c["D"], c["P"], causal=True, sm_scale=s["sm_scale"], num_pages=s["num_pages"])
    return s["plan"]


def _own_store(s):
    plan = _own_plan(s)
    plan.append_kv4(s["k_new"], s["v_new"], s["pool"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["binding"].attn_expand_kv4(s["pool"], s["page_ids"], s["case"]["D"], buf=s["back"], k_scale=s["k_scale"],
                                        v_scale=s["v_scale"])


def _own_decode4(s):
    return _own_plan(s).decode_kv4(s["q"], s["pool"], s["sinks"], s["out"], s["lse"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])


def _own_weights(s):
    c, plan = s["case"], _own_plan(s)
    if c["bits"] == 4:
        return plan.key_weights_kv4(s["q"], s["pool"], s["lse"], s["weights"], prev=s["prev"], decay=c["decay"],
                                    window=c["window"], k_scale=s["k_scale"])
    return plan.key_weights(s["q"], s["pool"], s["lse"], s["weights"], prev=s["prev"], decay=c["decay"],
                            window=c["window"])


def _own_evict(s):
    c, plan = s["case"], _own_plan(s)
    call = plan.evict_kv if c["bits"] == 16 else plan.evict_kv4
    call(s["weights"], s["pool"], c["budget"], c["recent"], kept=s["kept"], page_table_out=s["out_table"],
         kv_out=s["pool_out"], weights_out=s["weights_out"])
    if c["bits"] == 16:
        return s["kept"], s["pool_out"], s["weights_out"]
    back = s["binding"].attn_expand_kv4(s["pool_out"], s["out_table"], c["D"], buf=s["back"], k_scale=s["k_scale"],
                                        v_scale=s["v_scale"])
    return s["kept"], back, s["weights_out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "decode4": _own_decode4, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"store": _plain_store, "decode4": _plain_decode4, "weights": _plain_weights, "evict": _plain_evict}[op](state)


# --------------------------------------------------------- the same in 64 bits

def _two_to(k):
    """2 ** k for whole numbers k in -16 .. 16, without a rounding."""
    return torch.tensor([2.0 ** i for i in range(-16, 17)], dtype=torch.float64, device="cuda")[k + 16]


def _value4(block, P, D):
    """Values of one (page, K/V, head) block or several, from the bits of the two formats: fp64 [..., P, D]."""
    b = block.to(torch.int64)
    lead = b.shape[:-2]
    n = b[..., :8 * D]
    code = torch.stack((n % 16, n // 16), -1).reshape(*lead, P, D // GROUP, GROUP)
    e, m = (code // 2) % 4, code % 2
    mag = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * _two_to(e - 1))
    val = torch.where(code >= 8, -mag, mag)
    f = b[..., 8 * D:].reshape(*lead, P, D // GROUP)
    fe, fm = (f // 8) % 16, f % 8
    fs = torch.where(fe == 0, fm.double() / 512, (8 + fm.double()) * _two_to(fe - 10))
    fs = torch.where((fe == 15) & (fm == 7), torch.full_like(fs, float("nan")), fs) * torch.where(f >= 128, -1.0, 1.0)
    return (val * fs[..., None]).reshape(*lead, P, D)


def _nearest4(x):
    """What rows x (fp64, over the pool's scale) stand for once held in 4 bits."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    c = torch.arange(127, device=x.device)
    scales = torch.where(c < 8, c.double() / 512, (8 + (c % 8).double()) * _two_to(c // 8 - 10))
    out = torch.empty_like(x)
    flat, flat_out = x.reshape(-1, GROUP), out.view(-1, GROUP)
    for i in range(0, len(flat), 1 << 19):
        y = flat[i:i + (1 << 19)]
        want = y.abs().amax(-1) / 6
        hi = torch.searchsorted(scales, want).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = scales[hi] - want, want - scales[lo]
        s = scales[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)][:, None]
        far = (y.abs()[..., None] - grid * s[..., None]).abs()
        # Nearest, and of two equally near the one with the even code.
        best = far.amin(-1, keepdim=True)
        tie = (far == best) & ((torch.arange(8, device=x.device) % 2 == 0) | ((far == best).sum(-1, keepdim=True) == 1))
        flat_out[i:i + (1 << 19)] = torch.copysign(grid[tie.int().argmax(-1)] * s, y)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D, P, Hkv, G = case["D"], case["P"], case["Hkv"], case["Hq"] // case["Hkv"]
    kv, qo, h = _kv_lens(case), _qo_lens(case), s["host"]
    four = s["pool"].dtype == torch.uint8

    def table(b):
        return s["page_table"][h["kv_indptr"][b]:h["kv_indptr"][b + 1]].long()

    def half(b, which):                                # [kv_len, Hkv, D] of request b
        x = s["pool"][table(b), which]
        x = _value4(x, P, D) * (s["v_scale"] if which else s["k_scale"]) if four else x.double()
        return x.transpose(1, 2).reshape(-1, Hkv, D)[:kv[b]]

    if case["op"] == "store":
        new = torch.stack([_nearest4(s["k_new"].double() / s["k_scale"]) * s["k_scale"],
                           _nearest4(s["v_new"].double() / s["v_scale"]) * s["v_scale"]])   # [2, rows, Hkv, D]
        f = torch.tensor([s["k_scale"], s["v_scale"]], dtype=torch.float64, device="cuda")[:, None, None, None]
        out, at = torch.empty(s["back"].shape, dtype=torch.float64, device="cuda"), 0
        for b in range(len(kv)):
            n0 = kv[b] - qo[b]
            ids = table(b) if case["pages"] == "all" else table(b)[-1:]
            x = torch.cat([_value4(s["pool"][i], P, D)[None] * f for i in ids.split(1024)]) if len(ids) > 1024 else \
                _value4(s["pool"][ids], P, D) * f
            base = 0 if case["pages"] == "all" else (len(table(b)) - 1) * P
            t = torch.arange(max(n0, base), kv[b], device="cuda")
            x[(t - base) // P, :, :, t % P] = new[:, h["qo_indptr"][b] + t - n0].permute(1, 0, 2, 3)
            out[at:at + len(ids)] = x
            at += len(ids)
        return out

    if case["op"] == "decode4":
        outs, lses = [], []
        for b in range(len(kv)):
            q = s["q"][b].double().view(Hkv, G, D)
            x = torch.matmul(q, half(b, 0).permute(1, 2, 0)) * s["sm_scale"]              # [Hkv, G, T]
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"].double().view(Hkv, G, 1)], -1)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[..., None])[..., :kv[b]]
            outs.append(torch.matmul(p, half(b, 1).transpose(0, 1)).reshape(-1, D))
            lses.append(lse.reshape(-1))
        return torch.stack(outs), torch.stack(lses)

    if case["op"] == "weights":
        out, first = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda"), _first_rows(case)
        for b in range(len(kv)):
            k, r0, n0 = half(b, 0), h["qo_indptr"][b], kv[b] - qo[b]
            t = torch.arange(kv[b], device="cuda")
            w = torch.zeros(Hkv, kv[b], dtype=torch.float64, device="cuda")
            if case["decay"]:
                w[:, :n0] = case["decay"] * s["prev"][table(b)].transpose(0, 1).flatten(1)[:, :n0].double()
            for i in range(first[b], qo[b], 512):
                i1 = min(i + 512, qo[b])
                q = s["q"][r0 + i:r0 + i1].double().view(-1, Hkv, G, D).permute(1, 2, 0, 3)
                x = torch.matmul(q, k.permute(1, 2, 0)[:, None]) * s["sm_scale"]          # [Hkv, G, n, T]
                p = torch.exp(x - s["lse"][r0 + i:r0 + i1].double().view(-1, Hkv, G).permute(1, 2, 0)[..., None])
                see = t[None] <= (n0 + torch.arange(i, i1, device="cuda"))[:, None]
                w += (p * see).sum((1, 2))
            out[table(b)[t // P], :, t % P] = w.t()
        return out

    pool_out = torch.zeros(s["pool_out"].shape if not four else (len(s["pool_out"]), 2, Hkv, P, D), dtype=torch.float64,
                           device="cuda")
    w_out, kept, o = torch.zeros(s["weights_out"].shape, dtype=torch.float64, device="cuda"), [], s["out_indptr"].tolist()
    for b in range(len(kv)):
        n, m = kv[b], min(kv[b], case["budget"])
        w = s["weights"][table(b)].transpose(0, 1).flatten(1)[:, :n].double()            # [Hkv, n]
        new = max(0, n - case["recent"])
        # Position by rank: newest keys first, then by falling weight and rising index.
        group = torch.zeros_like(w)
        group[:, new:] = 1.0
        by_w = torch.argsort(-w, dim=-1, stable=True)
        rank = torch.gather(by_w, 1, torch.argsort(-torch.gather(group, 1, by_w), dim=-1, stable=True))
        src = rank[:, :m].sort(-1).values
        kept.append(torch.cat([src, torch.full((Hkv, case["budget"] - m), -1, device="cuda")], 1))
        dst = s["out_table"][o[b]:o[b + 1]].long()
        j = torch.arange(m, device="cuda")
        pick = src.t()
        for which in (0, 1):
            x = torch.gather(half(b, which), 0, pick[..., None].expand(-1, -1, D))
            pool_out[dst[j // P], which, :, j % P] = x
        w_out[dst[j // P], :, j % P] = torch.gather(w.t(), 0, pick)
    back = pool_out[s["out_table"].long()] if four else pool_out
    return torch.stack(kept), back, w_out
