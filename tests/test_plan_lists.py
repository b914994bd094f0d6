"""What a plan holds for key weights (CPU): its size follows the rows of the
batch, not the tiles of the contexts before them, so that planning a few rows
on long contexts (drafts to verify, chunks) costs what it did without."""
import pytest

from test_abi import OK, lib, plan   # noqa: F401  (lib: the built library's fixture)


def workspace(lib, qo, kv, causal=1):   # noqa: F811
    st, h, ws = plan(lib, qo, [k // 16 for k in kv], [16] * len(kv), causal=causal)
    assert st == OK
    lib.attn_plan_destroy(h)
    return int(getattr(ws, "value", ws))


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("batch,rows,long", [(16, 4, 131072), (64, 4, 32768), (256, 4, 16384), (16, 40, 131072)])
def test_few_rows_on_long_contexts_need_little(lib, batch, rows, long, causal):   # noqa: F811
    # One 4-byte entry per 32 tiles of 128 keys, and 256-byte rounding of the regions.
    more = workspace(lib, [rows] * batch, [long] * batch, causal) - workspace(lib, [rows] * batch, [1024] * batch, causal)
    assert more <= batch * (long - 1024) // (128 * 32) * 4 + 2048
