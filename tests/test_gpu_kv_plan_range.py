"""Page planning where a length leaves 32 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")


def test_a_length_past_32_bits_is_refused():
    """A table wide enough for 2^31 tokens and more: lengths and positions are
    32-bit numbers, so a request that would pass 2^31 - 1 is refused whole."""
    page, width, top = 1024, (1 << 21) + 2, 2**31 - 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, new = i32([top - 2, top - 2, top, 5]), i32([3, 2, 0, 1])
    table = torch.zeros(4, width, dtype=torch.int32, device="cuda")
    p = nv.kv_plan(ctx, new, table, i32([3, 1, 2, 0]), i32([4]), page_size=page, num_pages=4, tokens=6)
    assert p.seq_lens.tolist() == [top - 2, top, top, 6] and int(p.refused) == 1 and int(p.free_count) == 4
    assert p.slots.tolist() == [-1, -1, -1, page - 3, page - 2, 5]
    assert p.positions.tolist()[3:] == [top - 2, top - 1, 5]
    assert not table.any()
    # one page more than 2^31 tokens take is not taken
    p = nv.kv_plan(i32([top - 1]), i32([5]), table[:1], i32([3, 1, 2, 0]), i32([4]), page_size=page, num_pages=4, tokens=5)
    assert int(p.refused) == 1 and int(p.free_count) == 4 and p.slots.tolist() == [-1] * 5 and not table.any()
