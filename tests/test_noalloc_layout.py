"""attn_decode_noalloc's static array holds the decode regions of a plan's
workspace from its first byte on (CPU: reads the source): no pointer is formed
in front of it, and nothing on this path knows of the lists that only other
calls read."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_attention_sink_gb300", "csrc")


def test_scratch_starts_at_its_first_byte():
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "noalloc.cu")).read())
    assert re.findall(r"scratch\s*-|-\s*L\.\w+", re.sub(r"L\.part_lse - L\.counters", "", source)) == []
    assert not re.search(r"\blists|requests|weight_tiles", source)


def test_layout_of_the_decode_regions_starts_with_the_units():
    header = open(os.path.join(CSRC, "attn_internal.h")).read()
    fields = re.search(r"struct WorkspaceLayout \{(.*?)\};", header, re.S).group(1)
    assert re.findall(r"(\w+) = 0", fields)[0] == "units"
    with open(os.path.join(CSRC, "plan.cpp")) as plan:
        assert plan.read().count("size_t off = 0;\n    L.units = off;") == 2      # host and graph plans
