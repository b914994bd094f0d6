"""Cases of the operators around the attention calls, for measuring them.

  rope    rotary positions with one to four axes: a step's q and k rows turned,
          and (``cache``) the turned k and the v written into their pages
  pages   the cache's pages handed about: forked for samples and beams, cloned,
          and compacted to the front of the pools
  cross   cross attention: the rows of each sequence over all of an encoder's
          states, which have a length of their own

``run`` computes an operator in elementary torch operations, or, where ``own``
is set, through the library's entry points on the same inputs.

Pair i of a row turns by the angle positions[axis[i]] * inv_freq[i].  A page is
free where its count in ``refs`` is 0; new pages are the lowest free ones.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    gptoss = dict(Hq=64, Hkv=8, D=64, P=16)
    qwen = dict(Hq=64, Hkv=4, D=128, P=64)
    return [
        # One decode step of a serving batch: q turned, k turned into its page, v beside it.
        dict(name="rope_step", op="rope", cache=True, batch=64, kv_lo=1024, kv_hi=8192, lens=0, qo=1, rot=64, axes=1,
             woven=False, inter=False, inverse=False, scale=1.0, **gptoss),
        # Prompts of text and images (time, height, width), rows as the fused projection leaves them.
        dict(name="rope_prompts", op="rope", cache=True, batch=5, kv_lo=1500, kv_hi=8192, lens=1, qo=0, rot=128, axes=3,
             woven=False, inter=False, inverse=False, scale=1.0, **qwen),
        # An image encoder's patches (height, width); no cache.
        dict(name="rope_patches", op="rope", cache=False, batch=3, kv_lo=1021, kv_hi=4096, lens=2, qo=0, rot=64, axes=2,
             woven=False, inter=False, inverse=False, scale=1.0, Hq=16, Hkv=16, D=64, P=16),
        # The gradient's way back through it: neighbouring dims paired, half of each head turned, axes interwoven.
        dict(name="rope_back", op="rope", cache=False, batch=4, kv_lo=900, kv_hi=4096, lens=3, qo=0, rot=64, axes=3,
             woven=True, inter=True, inverse=True, scale=1.25, Hq=32, Hkv=8, D=128, P=16),
        # Two samples more for some requests of a step.
        dict(name="fork_step", op="pages", do="fork", batch=64, children=32, kv_lo=1024, kv_hi=8192, lens=4, layers=2,
             used=0.8, **gptoss),
        # Beam search over a large batch: every request's beams are forked anew.
        dict(name="fork_beams", op="pages", do="fork", batch=128, children=1024, kv_lo=512, kv_hi=4096, lens=5, layers=3,
             used=0.8, **qwen),
        # A prefix's pages copied for a request that will write into them.
        dict(name="clone_prefix", op="pages", do="clone", batch=40, children=301, kv_lo=512, kv_hi=4096, lens=6, layers=2,
             used=0.5, **gptoss),
        # After a night of traffic: what is used moves to the front of the pools.
        dict(name="compact", op="pages", do="compact", batch=80, children=0, kv_lo=1024, kv_hi=8192, lens=7, layers=2,
             used=0.6, **gptoss),
        # The smallest call: single rows over short texts.
        dict(name="cross_tiny", op="cross", batch=2, qo_lo=1, qo_hi=1, kv_lo=40, kv_hi=77, lens=8, padded=True, fused=False,
             sinks=False, Hq=8, Hkv=2, D=64),
        # A step of a speech decoder: five beams on each recording's states, every query head with its own KV head.
        dict(name="cross_beams", op="cross", batch=48, qo_lo=5, qo_hi=5, kv_lo=1500, kv_hi=1500, lens=9, padded=True,
             fused=True, sinks=False, Hq=16, Hkv=16, D=64),
        # A step over long documents or videos, sixteen query heads on each KV head.
        dict(name="cross_long", op="cross", batch=16, qo_lo=1, qo_hi=1, kv_lo=2048, kv_hi=32768, lens=10, padded=False,
             fused=False, sinks=True, Hq=64, Hkv=4, D=128),
        # Prompts over images' states; some sequences have none.
        dict(name="cross_prompts", op="cross", batch=9, qo_lo=200, qo_hi=2048, kv_lo=0, kv_hi=6404, lens=11, padded=False,
             fused=True, sinks=True, Hq=64, Hkv=8, D=64),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "pages", "pages", "cross", "cross", "cross"])
    D = rng.choice([64, 128])
    P = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16])
    Hq = Hkv * G
    kv_hi = _spread(rng, 2, 32768)
    kv_lo = max(1, int(kv_hi * rng.uniform(0.05, 1.0)))
    lens = rng.randrange(1 << 20)
    heads = dict(Hq=Hq, Hkv=Hkv, D=D)
    if op == "rope":
        cache = rng.random() < 0.6
        while kv_hi * (Hq + 2 * Hkv) * D > 1 << 27:
            kv_hi = kv_hi // 2 + 1
        kv_lo = min(kv_lo, kv_hi)
        qo = rng.choice([0, 1, 1, _spread(rng, 1, kv_hi)])
        rows = kv_hi if qo == 0 else min(qo, kv_hi)
        batch = max(1, min(_spread(rng, 1, 256), (1 << 27) // (rows * (Hq + 2 * Hkv) * D), (1 << 28) // (kv_hi * Hkv * D)))
        return dict(op=op, cache=cache, batch=batch, kv_lo=kv_lo, kv_hi=kv_hi, lens=lens, qo=qo, P=P,
                    rot=rng.choice([D, D, D // 2, 16, D - 16]), axes=rng.randint(1, 4), woven=rng.random() < 0.3,
                    inter=rng.random() < 0.4, inverse=not cache and rng.random() < 0.5,
                    scale=rng.choice([1.0, 1.0, 1.25]), **heads)
    if op == "pages":
        do = rng.choice(["fork", "clone", "compact"])
        layers = rng.randint(1, 3)
        kv_hi = max(2, min(kv_hi, 8192, (1 << 28) // (Hkv * D * layers)))
        kv_lo = min(kv_lo, kv_hi)
        batch = max(1, min(_spread(rng, 1, 128), (1 << 27) // (kv_hi * Hkv * D * layers)))
        children = max(1, min(_spread(rng, 1, 1024), (1 << 26) // (P * Hkv * D * layers)))
        return dict(op=op, do=do, batch=batch, children=children, kv_lo=kv_lo, kv_hi=kv_hi, lens=lens, layers=layers,
                    used=rng.uniform(0.2, 0.95), P=P, **heads)
    kv_lo = rng.choice([0, kv_lo, kv_hi])
    qo_hi = rng.choice([1, rng.randint(2, 16), _spread(rng, 2, 2048)])
    while Hq * qo_hi * kv_hi > 1 << 28 and qo_hi > 1:
        qo_hi = qo_hi // 2 + 1
        kv_hi = kv_hi // 2 + 1
        kv_lo = min(kv_lo, kv_hi)
    batch = max(1, min(_spread(rng, 1, 128), (1 << 29) // (Hq * qo_hi * kv_hi), (1 << 28) // (kv_hi * Hkv * D),
                       (1 << 26) // (qo_hi * Hq * D)))
    return dict(op=op, batch=batch, qo_lo=rng.choice([0, 1, qo_hi]), qo_hi=qo_hi, kv_lo=kv_lo, kv_hi=kv_hi, lens=lens,
                padded=rng.random() < 0.5, fused=rng.random() < 0.5, sinks=rng.random() < 0.5, **heads)


def _lengths(case, lo, hi, salt):
    """The case's lengths, the shortest and the longest allowed among them."""
    rng = random.Random(case["lens"] * 8 + salt)
    lens = [rng.randint(lo, hi) for _ in range(case["batch"])]
    lens[0] = hi
    if len(lens) > 1:
        lens[1] = lo
    return lens


def _kv_lens(case):
    return _lengths(case, case["kv_lo"], case["kv_hi"], 0)


def _qo_lens(case):
    if case["op"] == "cross":
        return _lengths(case, case["qo_lo"], case["qo_hi"], 1)
    return [n if case["qo"] == 0 else min(case["qo"], n) for n in _kv_lens(case)]


def _csr(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _pages_of(lens, P):
    return [(n + P - 1) // P for n in lens]


def _parents(case):
    rng = random.Random(case["lens"] * 8 + 2)
    return [rng.randrange(case["batch"]) for _ in range(case["children"])]


def _pages_moved(case):
    """Pages whose contents a pass copies, as far as the sizes tell."""
    kv, P = _kv_lens(case), case["P"]
    if case["do"] == "fork":
        return sum(kv[p] % P != 0 for p in _parents(case))
    if case["do"] == "clone":
        return min(case["children"], sum(_pages_of(kv, P)))
    return int(sum(_pages_of(kv, P)) * (1 - case["used"]))     # the used share of what lies behind


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        rows = sum(_qo_lens(case))
        heads = Hq + Hkv + (Hkv if case["cache"] else 0)
        return {"bytes": rows * (4 * D * heads + 4 * case["axes"] + (8 if case["cache"] else 0)),
                "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    if case["op"] == "pages":
        kv, P = _kv_lens(case), case["P"]
        num_pages = int(sum(_pages_of(kv, P)) / case["used"]) + 1
        page = 4 * Hkv * P * D
        entries = {"fork": sum(_pages_of([kv[p] for p in _parents(case)], P)) if case["do"] == "fork" else 0,
                   "clone": case["children"], "compact": sum(_pages_of(kv, P))}[case["do"]]
        return {"bytes": 2 * case["layers"] * _pages_moved(case) * page + 4 * num_pages + 16 * entries, "flops": num_pages}
    kv, qo = _kv_lens(case), _qo_lens(case)
    return {"bytes": 4 * D * Hkv * sum(n for n, m in zip(kv, qo) if m) + sum(qo) * Hq * (4 * D + 4),
            "flops": 4 * D * Hq * sum(n * m for n, m in zip(kv, qo))}


# ------------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rope_tables(case):
    """Frequencies and axes of a row's pairs (host lists): sections in order, or interwoven."""
    half, axes = case["rot"] // 2, case["axes"]
    freq = torch.tensor([10000.0 ** (-2 * i / case["rot"]) for i in range(half)], dtype=torch.float64)
    if case["woven"]:
        axis = [i % axes for i in range(half)]
    else:
        first = half // 4 if axes == 3 else half // axes     # time takes a quarter, height and width share the rest
        ends = [first + (half - first) * a // max(1, axes - 1) for a in range(axes)]
        axis = [min(axes - 1, sum(i >= e for e in ends)) for i in range(half)]
    return [float(f) for f in freq.float()], axis


def _prepare_rope(case, g, s):
    D, Hq, Hkv, P, axes = case["D"], case["Hq"], case["Hkv"], case["P"], case["axes"]
    kv, qo = _kv_lens(case), _qo_lens(case)
    rows, i32 = sum(qo), dict(dtype=torch.int32, device="cuda")
    qkv = _normal(g, rows, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
    heads = qkv.view(rows, Hq + 2 * Hkv, D)
    s["q"], s["k"], s["v"] = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
    at = torch.cat([torch.arange(n - m, n) for n, m in zip(kv, qo)]).cuda()
    pos = at[None].repeat(axes, 1)
    if axes > 1:     # inside images, the place in the grid comes on top
        grid = torch.randint(0, 64, (axes - 1, rows), device="cuda", generator=g)
        pos[1:] += grid * ((at // 256) % 2)
    s["positions"] = pos.to(torch.int32)
    s["inv_freq"], s["axis"] = _rope_tables(case)
    s["q_out"] = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    if not case["cache"]:
        s["k_out"] = torch.zeros(rows, Hkv, D, dtype=torch.bfloat16, device="cuda")
        return
    n_pages = _pages_of(kv, P)
    total = sum(n_pages)
    s["num_pages"] = num_pages = total + max(1, total // 4)
    s["page_table"] = torch.randperm(num_pages, device="cuda", generator=g)[:total].to(torch.int32)
    s["host"] = dict(qo_indptr=_csr(qo), kv_indptr=_csr(n_pages), last_page_len=[n - (p - 1) * P for n, p in zip(kv, n_pages)])
    s["pool"] = torch.zeros(num_pages, 2, Hkv, P, D, dtype=torch.bfloat16, device="cuda")
    first = torch.tensor(s["host"]["kv_indptr"][:-1], device="cuda").repeat_interleave(torch.tensor(qo, device="cuda"))
    s["page"], s["row"] = s["page_table"][first + at // P].long(), at % P


def _prepare_pages(case, g, s):
    D, Hkv, P, do = case["D"], case["Hkv"], case["P"], case["do"]
    kv = _kv_lens(case)
    n_pages = _pages_of(kv, P)
    total = sum(n_pages)
    parents = _parents(case) if do == "fork" else []
    fresh = sum(kv[p] % P != 0 for p in parents) if do == "fork" else min(case["children"], total) if do == "clone" else 0
    s["num_pages"] = num_pages = max(int(total / case["used"]) + 1, total + fresh)
    i32 = dict(dtype=torch.int32, device="cuda")
    s["page_table"] = torch.randperm(num_pages, device="cuda", generator=g)[:total].to(torch.int32)
    s["kv_indptr"] = torch.tensor(_csr(n_pages), **i32)
    s["kv_lens"] = torch.tensor(kv, **i32)
    s["refs"] = torch.zeros(num_pages, **i32)
    s["refs"][s["page_table"].long()] = 1
    s["pools"] = [_normal(g, num_pages, Hkv * P * D).to(torch.bfloat16).repeat(1, 2).view(num_pages, 2, Hkv, P, D)
                  for _ in range(case["layers"])]
    # The children (clones) of the step before, which the pass gives up first.
    if do == "fork":
        s["parents"] = torch.tensor(parents, **i32)
        s["entries"] = sum(n_pages[p] for p in parents)
        s["old"], _ = _plain_fork(s)
    elif do == "clone":
        s["src"] = s["page_table"][:fresh].contiguous()
        s["old"] = _plain_alloc(s["refs"], fresh)
        s["refs"][s["old"].long()] = 1
    else:
        s["refs0"], s["table0"] = s["refs"].clone(), s["page_table"].clone()


def _prepare_cross(case, g, s):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    kv, qo = _kv_lens(case), _qo_lens(case)
    room = case["kv_hi"] if case["padded"] else 0         # rows of the states that each sequence takes
    s["kv_start"] = [b * room for b in range(len(kv))] if case["padded"] else _csr(kv)[:-1]
    s["kv_len"], s["qo_indptr"] = kv, _csr(qo)
    s["kv_rows"] = rows = max(1, room * len(kv) if case["padded"] else sum(kv))
    s["q"] = _normal(g, sum(qo), Hq, D).to(torch.bfloat16)
    both = _normal(g, rows, 2 * Hkv, D)
    both[:, :Hkv] *= torch.exp(0.4 * _normal(g, Hkv, D))  # K channels of uneven size
    both = both.to(torch.bfloat16)
    if case["padded"]:                                    # what lies behind a sequence is not read
        for b, n in enumerate(kv):
            both[b * room + n:(b + 1) * room] = float("nan")
    s["k"], s["v"] = both[:, :Hkv], both[:, Hkv:]
    if not case["fused"]:
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    s["sinks"] = _normal(g, Hq) if case["sinks"] else None
    s["sm_scale"] = D ** -0.5
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(len(s["q"]), Hq, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    {"rope": _prepare_rope, "pages": _prepare_pages, "cross": _prepare_cross}[case["op"]](case, g, s)
    return s


# -------------------------------------------------------------- plain forms

def _plain_turned(x, cos, sin, inter):
    """x [rows, H, D] with its first 2 * cos.shape[-1] dims turned."""
    x = x.float()
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    c, s = cos[:, None], sin[:, None]
    y, z = a * c - b * s, a * s + b * c
    both = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((both, x[..., 2 * half:]), -1)


def _plain_rope(s):
    c = s["case"]
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    angle = s["positions"][s["axis"]].t().double() * freq          # [rows, pairs]; far positions need the bits
    if c["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float() * c["scale"], torch.sin(angle).float() * c["scale"]
    s["q_out"].copy_(_plain_turned(s["q"], cos, sin, c["inter"]))
    k = _plain_turned(s["k"], cos, sin, c["inter"]).to(torch.bfloat16)
    if not c["cache"]:
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    s["pool"][s["page"], 0, :, s["row"]] = k
    s["pool"][s["page"], 1, :, s["row"]] = s["v"]
    return s["q_out"], s["pool"]


def _plain_alloc(refs, n):
    return (refs == 0).nonzero()[:n, 0].to(torch.int32)


def _count(refs, ids, by):
    refs.index_add_(0, ids.long(), torch.full_like(ids, by))


def _plain_fork(s):
    P, parents, indptr = s["case"]["P"], s["parents"].long(), s["kv_indptr"].long()
    n = indptr[1:] - indptr[:-1]
    out_indptr = torch.nn.functional.pad(n[parents].cumsum(0), (1, 0))
    child = torch.repeat_interleave(torch.arange(len(parents), device="cuda"), n[parents], output_size=s["entries"])
    table = s["page_table"][indptr[parents][child] + torch.arange(s["entries"], device="cuda") - out_indptr[child]]
    part = s["kv_lens"].long()[parents] % P != 0                   # whose last page is not full
    at = out_indptr[1:][part] - 1
    src = table[at]
    _count(s["refs"], table, 1)
    _count(s["refs"], src, -1)
    dst = _plain_alloc(s["refs"], len(src))
    s["refs"][dst.long()] = 1
    table[at] = dst
    for pool in s["pools"]:
        pool[dst.long()] = pool[src.long()]
    return table, out_indptr.to(torch.int32)


def _plain_pages(s):
    do, refs, pools = s["case"]["do"], s["refs"], s["pools"]
    if do == "fork":
        _count(refs, s["old"], -1)
        s["old"], indptr = _plain_fork(s)
        return [s["old"], indptr, refs, *pools]
    if do == "clone":
        _count(refs, s["old"], -1)
        s["old"] = ids = _plain_alloc(refs, len(s["src"]))
        _count(refs, ids, 1)
        for pool in pools:
            pool[ids.long()] = pool[s["src"].long()]
        return [ids, refs, *pools]
    refs.copy_(s["refs0"])                                         # the scheduler's tables of this step
    s["page_table"].copy_(s["table0"])
    used = refs > 0
    front = torch.arange(len(refs), device="cuda") < used.sum()
    dst, src = (front & ~used).nonzero()[:, 0], (~front & used).nonzero()[:, 0].flip(0)
    remap = torch.where(used, torch.arange(len(refs), device="cuda"), -1)
    remap[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    for pool in pools:
        pool[dst] = pool[src]
    s["page_table"].copy_(remap[s["page_table"].long()])
    return [s["page_table"], remap.to(torch.int32), refs, *pools]


def _plain_cross(s):
    c, h = s["case"], s["qo_indptr"]
    Hkv, G, D = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    for b, (start, n) in enumerate(zip(s["kv_start"], s["kv_len"])):
        r0, r1 = h[b], h[b + 1]
        if r0 == r1:
            continue
        step = max(1, (1 << 28) // max(1, c["Hq"] * n))
        k, v = s["k"][start:start + n].float().permute(1, 2, 0), s["v"][start:start + n].float().transpose(0, 1)
        for r in range(r0, r1, step):
            e = min(r + step, r1)
            q = s["q"][r:e].float().view(e - r, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
            x = torch.matmul(q, k) * s["sm_scale"]                  # [Hkv, rows * G, T]
            sink = x.new_full((Hkv, (e - r) * G, 1), float("-inf")) if s["sinks"] is None else \
                s["sinks"].view(Hkv, 1, G).expand(-1, e - r, -1).reshape(Hkv, -1, 1)
            x = torch.cat((x, sink), -1)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p[..., :n], v) / torch.where(total == 0, torch.ones_like(total), total)
            s["out"][r:e] = o.view(Hkv, e - r, G, D).permute(1, 0, 2, 3).reshape(e - r, -1, D).to(torch.bfloat16)
            s["lse"][r:e] = (m + total.log()).view(Hkv, e - r, G).permute(1, 0, 2).reshape(e - r, -1)
    return s["out"], s["lse"]


# ---------------------------------------------------- the library's operators

def _binding(s):
    if "binding" not in s:
        from paged_kv_attention_sink_gb300 import binding
        s["binding"] = binding
    return s["binding"]


def _own_rope(s):
    c, lib = s["case"], _binding(s)
    if "rope" not in s:      # kept with the model, and the plan with the batch
        s["rope"] = lib.Rope(s["inv_freq"], axis=s["axis"], interleaved=c["inter"], scale=c["scale"])
        if c["cache"]:
            h = s["host"]
            s["plan"] = lib.Plan(h["qo_indptr"], h["kv_indptr"], s["page_table"], h["last_page_len"], c["Hq"], c["Hkv"],
                                 c["D"], c["P"], num_pages=s["num_pages"])
    if c["cache"]:
        s["plan"].append_kv_rope(s["rope"], s["positions"], s["q"], s["k"], s["v"], s["pool"], q_out=s["q_out"])
        return s["q_out"], s["pool"]
    return s["rope"].apply(s["positions"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], inverse=c["inverse"])


def _own_pages(s):
    do, lib = s["case"]["do"], _binding(s)
    if "pages" not in s:     # kept with the cache
        s["pages"] = lib.PagePool(s["pools"], s["case"]["P"], refs=s["refs"])
    pages = s["pages"]
    if do == "fork":
        pages.free(s["old"])
        s["old"], indptr = pages.fork(s["page_table"], s["kv_indptr"], s["kv_lens"], s["parents"], s["entries"])
        return [s["old"], indptr, s["refs"], *s["pools"]]
    if do == "clone":
        pages.free(s["old"])
        s["old"] = ids = pages.alloc(len(s["src"]))
        pages.copy(s["src"], ids)
        return [ids, s["refs"], *s["pools"]]
    s["refs"].copy_(s["refs0"])
    s["page_table"].copy_(s["table0"])
    remap = pages.compact(s["page_table"])
    return [s["page_table"], remap, s["refs"], *s["pools"]]


def _own_cross(s):
    c = s["case"]
    if "plan" not in s:      # made once per batch; every layer uses it
        s["plan"] = _binding(s).CrossPlan(s["qo_indptr"], s["kv_start"], s["kv_len"], s["kv_rows"], c["Hq"], c["Hkv"],
                                          c["D"], sm_scale=s["sm_scale"])
    return s["plan"].attend(s["q"], s["k"], s["v"], s["sinks"], s["out"], s["lse"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "pages": _own_pages, "cross": _own_cross}[op](state)
    return {"rope": _plain_rope, "pages": _plain_pages, "cross": _plain_cross}[op](state)


# --------------------------------------------------------- the same in 64 bits

def _exact_rope(case, s):
    rot, pairs = case["rot"], case["rot"] // 2
    first = [2 * i if case["inter"] else i for i in range(pairs)]
    second = [2 * i + 1 if case["inter"] else i + pairs for i in range(pairs)]
    angle = torch.stack([s["positions"][a].double() * f for a, f in zip(s["axis"], s["inv_freq"])], 1)
    turn = torch.polar(torch.full_like(angle, case["scale"]), -angle if case["inverse"] else angle)

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if not case["cache"]:
        return turned(s["q"]), turned(s["k"])
    pool = torch.zeros(s["pool"].shape, dtype=torch.float64, device="cuda")
    pool[s["page"], 0, :, s["row"]] = turned(s["k"])
    pool[s["page"], 1, :, s["row"]] = s["v"].double()
    return turned(s["q"]), pool


def _exact_pages(case, s):
    """Page by page on the host."""
    P, do = case["P"], case["do"]
    refs, table = s["refs"].tolist(), s["page_table"].tolist()
    moves = {}                                             # page -> whose contents it gets
    if do == "compact":
        remap = [p if n else -1 for p, n in enumerate(refs)]
        low, high = 0, len(refs) - 1
        while True:
            while low < len(refs) and refs[low]:
                low += 1
            while high >= 0 and not refs[high]:
                high -= 1
            if low > high:
                break
            refs[low], refs[high] = refs[high], 0
            remap[high] = low
            moves[low] = high
        head = [[remap[p] for p in table], remap, refs]
    else:
        for p in s["old"].tolist():
            refs[p] -= 1
        empty = iter([p for p, n in enumerate(refs) if n == 0])
        if do == "clone":
            ids = []
            for p in s["src"].tolist():
                ids.append(next(empty))
                refs[ids[-1]] = 1
                moves[ids[-1]] = p
            head = [ids, refs]
        else:
            lens, start, out, indptr = s["kv_lens"].tolist(), s["kv_indptr"].tolist(), [], [0]
            for b in s["parents"].tolist():
                pages = table[start[b]:start[b + 1]]
                if lens[b] % P:
                    moves[new := next(empty)] = pages[-1]
                    pages[-1] = new
                for p in pages:
                    refs[p] += 1
                out += pages
                indptr.append(len(out))
            head = [out, indptr, refs]
    where = torch.arange(len(refs), device="cuda")
    where[list(moves)] = torch.tensor(list(moves.values()), device="cuda", dtype=torch.long)
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in head] + [pool[where] for pool in s["pools"]]


def _exact_cross(case, s):
    G, outs, lses = case["Hq"] // case["Hkv"], [], []
    for b, (start, n) in enumerate(zip(s["kv_start"], s["kv_len"])):
        q = s["q"][s["qo_indptr"][b]:s["qo_indptr"][b + 1]].double()
        out, lse = torch.zeros_like(q), torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            k, v = s["k"][start:start + n, h // G].double(), s["v"][start:start + n, h // G].double()
            for r in range(0, len(q), 512):
                x = q[r:r + 512, h] @ k.t() * s["sm_scale"]
                if s["sinks"] is not None:
                    x = torch.cat((s["sinks"][h].double().expand(len(x), 1), x), 1)
                if x.shape[1]:
                    lse[r:r + 512, h] = torch.logsumexp(x, 1)
                    out[r:r + 512, h] = torch.exp(x - lse[r:r + 512, h, None])[:, x.shape[1] - n:] @ v
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "pages": _exact_pages, "cross": _exact_cross}[case["op"]](case, s)
