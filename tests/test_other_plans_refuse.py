"""Ragged and graph plans refuse the compressed cache's methods with a
TypeError, those that only read the plan among them (CPU: no plan is made)."""
import os

import pytest

from paged_kv_attention_sink_gb300 import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.LIB), reason="libattn.so is not built")

READS = {"kv_lens": lambda p: p.kv_lens, "evicted_lens": lambda p: p.evicted_lens(4)}
CALLS = ["append_kv", "append_kv4", "decode_kv4", "key_weights", "key_weights_kv4", "evict_kv", "evict_kv4"]


@pytest.mark.parametrize("kind", ["RaggedPlan", "GraphPlan"])
@pytest.mark.parametrize("name", [*READS, *CALLS])
def test_refused(kind, name):
    from paged_kv_attention_sink_gb300 import binding
    plan = object.__new__(getattr(binding, kind))
    with pytest.raises(TypeError):
        READS[name](plan) if name in READS else getattr(plan, name)()


def test_a_ragged_plan_has_no_4_bit_cache():
    from paged_kv_attention_sink_gb300 import binding
    with pytest.raises(TypeError):
        object.__new__(binding.RaggedPlan).kv4_shape()
