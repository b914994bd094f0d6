"""The README's example of the operators around attention runs as it stands."""
import os
import re

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_example():
    from paged_kv_attention_sink_gb300 import binding
    section = open(README).read().split("### Around attention")[1]
    block = re.search(r"```python\n(.*?)```", section, re.S).group(1)
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    # A prompt of 90 tokens on six pages of 16; 5 and 3 rows over 40 and 300 states.
    rows, Hq, Hkv, D, P = 90, 16, 4, 64, 16
    n_pages = -(-rows // P)
    qkv = randn(rows, Hq + 2 * Hkv, D)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    names = dict(
        binding=binding, torch=torch, q=q, k=k, v=v, dq=randn(rows, Hq, D), dk=randn(rows, Hkv, D),
        inv_freq=1000.0 ** (-np.arange(D // 2) / (D // 2)), axis=[p % 3 for p in range(D // 2)],
        positions=torch.randint(0, 100, (3, rows), generator=g, **i32), kv_cache=torch.zeros(n_pages, 2, Hkv, P, D,
                                                                                             dtype=torch.bfloat16, device="cuda"),
        plan=binding.Plan([0, rows], [0, n_pages], torch.arange(n_pages, **i32), [rows - (n_pages - 1) * P], Hq, Hkv, D, P,
                          num_pages=n_pages),
        kv_layer0=randn(40, 2, Hkv, P, D), kv_layer1=randn(40, 2, Hkv, P, D),
        kv_indptr=torch.tensor([0, 5, 12], **i32), kv_lens=torch.tensor([70, 112], **i32), parents=torch.tensor([1, 0, 1], **i32),
        child_pages=7 + 5 + 7, qo_indptr=[0, 50, rows], kv_start=[0, 40], kv_len=[40, 300], kv=randn(340, 2 * 16, D))
    exec(block, names)
    assert names["q"].shape == (rows, Hq, D) and names["kv_cache"].any() and names["dk"].shape == (rows, Hkv, D)
    assert names["child_indptr"].tolist() == [0, 7, 12, 19]
    # seven full pages shared by two children, four by one, and a copy of the last one
    assert sorted(names["pages"].refs.tolist(), reverse=True)[:13] == [2] * 7 + [1] * 5 + [0]
    assert sorted(set(names["child_table"].tolist())) == list(range(12))
    assert names["out"].shape == (rows, 16, D) and names["lse"].shape == (rows, 16) and bool(torch.isfinite(names["lse"]).all())
    for x in ("plan", "pages", "cross"):
        assert names[x].device_error() == 0
