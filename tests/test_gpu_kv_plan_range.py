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


def test_requests_past_the_steps_tokens_are_refused():
    """`tokens` says how many new tokens the step has room for: a request that
    does not fit whole takes no page, where part of it would have no slot and
    its table no entry for the pages taken."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, new, free, count = i32([3, 16, 0, 20]), i32([5, 40, 3, 0]), i32([4, 5, 6, 7] + [0] * 4), i32([4])
    table = torch.full((4, 6), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[1, 0], table[3, :2] = 0, 1, i32([2, 3])
    for tokens, lens, left in ((10, [8, 16, 0, 20], 4), (45, [8, 56, 0, 20], 1), (47, [8, 56, 0, 20], 1), (48, [8, 56, 3, 20], 0)):
        t = table.clone()
        p = nv.kv_plan(ctx, new, t, free, count, page_size=16, num_pages=8, tokens=tokens)
        assert p.seq_lens.tolist() == lens and int(p.free_count) == left, tokens
        assert int(p.refused) == sum(a + b != n for a, b, n in zip([3, 16, 0, 20], [5, 40, 3, 0], lens))
        assert p.cu_new.tolist() == [0, 5, 45, 48, 48]
        for b, n in enumerate(lens):  # a page for every token that a length counts
            assert (t[b, :-(-n // 16)] >= 0).all(), (tokens, b)
        slots = p.slots.tolist()
        assert all(s >= 0 for s in slots[:5]) and all((s >= 0) == (lens[1] == 56) for s in slots[5:45])
        assert all((s >= 0) == (lens[2] == 3) for s in slots[45:48])


def test_running_totals_stay_in_32_bits():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    top = 2**31 - 1
    p = nv.kv_plan(i32([0, 0, 0, 4]), i32([3, top, top, 0]), torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                   i32([1, 2]), i32([2]), page_size=16, num_pages=2, tokens=3)
    assert p.cu_new.tolist() == [0, 3, top, top, top] and p.seq_lens.tolist() == [3, 0, 0, 4]
    assert int(p.refused) == 2 and int(p.free_count) == 1
