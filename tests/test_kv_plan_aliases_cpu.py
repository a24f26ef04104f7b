"""nvfp4_kv_plan refuses outputs that are its inputs: its workgroups read the
inputs while another one writes the outputs.  No GPU needed."""
import pytest

from nvfp4_block_scaled_02_amd import _native as N

INPUTS = ("ctx_lens", "new_lens", "free_pages", "free_count", "block_table")
OUTPUTS = ("cu_new", "seq_lens", "positions", "slots", "free_count_out", "refused")


def _args(**kw):
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(INPUTS + OUTPUTS)}  # never dereferenced
    return N.KVPlanArgs(**{**at, **dict(batch=3, table_width=8, num_pages=10, page_size=16, tokens=5), **kw})


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("inp", INPUTS)
def test_an_output_that_is_an_input(out, inp):
    a = _args()
    assert N.lib().nvfp4_kv_plan(_args(**{out: getattr(a, inp)}), None) == N.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(ctx_lens=None), dict(new_lens=None), dict(seq_lens=None), dict(block_table=None),
    dict(positions=None), dict(slots=None), dict(free_pages=None), dict(free_count=None),
    dict(cu_new=None), dict(free_count_out=None), dict(refused=None), dict(batch=-1),
    dict(tokens=-1), dict(table_width=-1), dict(batch=1 << 31), dict(tokens=1 << 31),
    dict(table_width=1 << 31), dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=4),
    dict(page_size=48), dict(page_size=2048), dict(page_size=0), dict(slots=0x900004),
    dict(ctx_lens=0x100001), dict(refused=0xB00002), dict(batch=1 << 30, table_width=1 << 30),
])
def test_other_refusals_with_buffers_apart(kw):
    assert N.lib().nvfp4_kv_plan(_args(**kw), None) == N.ERR_INVALID
