"""Page planning on the device against the plain loop: whole numbers, exact."""
import numpy as np
import pytest

import kv_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")


def _run(ctx, new, width, page, pages, count=None, pad=0, bad=False, seed=0):
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(ctx), width), -7, np.int32)
    used = 0
    for b, c in enumerate(ctx):
        n = min(-(-max(int(c), 0) // page), width)
        table[b, :n] = order[(used + np.arange(n)) % pages]
        used += n
    if bad:
        table[rng.random(table.shape) < 0.3] = pages + 5
    free = rng.permutation(pages).astype(np.int32)
    count = pages if count is None else count
    tokens = int(np.maximum(new, 0).sum()) + pad
    want = R.plan(ctx, new, table, free, count, page, pages, tokens)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    tab = d(table)
    args = (d(ctx), d(new), tab, d(free), d(np.array([count], np.int32)))
    for _ in range(2):  # the inputs stay: a second call gives the same
        p = nv.kv_plan(*args, page_size=page, num_pages=pages, tokens=tokens)
        got = [t.cpu().numpy() for t in (p.cu_new, p.seq_lens, p.positions, p.slots, tab)]
        for g, w, n in zip(got, want, ("cu_new", "seq_lens", "positions", "slots", "block_table")):
            assert np.array_equal(g, w), n
        assert int(p.free_count.item()) == want[5] and int(p.refused.item()) == want[6]
    return want


@pytest.mark.parametrize("batch", [1, 3, 64, 1023, 1024, 1025, 2600])
@pytest.mark.parametrize("page", [8, 16, 128])
def test_mixed_batches(batch, page):
    rng = np.random.default_rng(batch * 1000 + page)
    ctx = rng.integers(0, 300, batch)
    new = np.where(rng.random(batch) < 0.3, rng.integers(0, 90, batch), 1)
    ctx[::7] = 0
    new[::11] = 0
    width = -(-400 // page)
    w = _run(ctx, new, width, page, pages=batch * width + 3, pad=int(rng.integers(0, 5)))
    assert w[6] == 0


def test_decode_step_and_page_borders():
    # one token each, at every place in a page: a new page exactly at its start
    _run(np.arange(40), np.ones(40), 8, 16, 200)
    _run([16, 15, 17, 0], [1, 1, 1, 1], 3, 16, 16)


@pytest.mark.parametrize("tokens", [1023, 1024, 1025, 70000])
def test_one_long_prompt(tokens):
    _run([5, 0], [tokens, 1], -(-(tokens + 8) // 16), 16, tokens // 16 + 9)


def test_too_few_pages_refuses_in_order():
    # 4 free pages: request 0 takes 3, request 1 needs 2, request 2 none, request 3 one
    w = _run([0, 0, 3, 16], [40, 20, 2, 1], 8, 16, 64, count=4)
    assert w[6] == 2 and w[5] == 1 and list(w[1]) == [40, 0, 5, 16]
    _run([0] * 1500, [20] * 1500, 4, 16, 4000, count=2101)
    _run([0], [1], 4, 16, 8, count=0)
    _run([0], [1], 4, 16, 8, count=-3)
    _run([0, 9], [1, 3], 4, 16, 8, count=1000)  # more than the pages: clamped


def test_longer_than_the_table_is_refused_and_takes_nothing():
    w = _run([0, 10, 40], [100, 5, 100], 4, 16, 64)
    assert w[6] == 2 and list(w[1]) == [0, 15, 40]
    _run([500, 1], [1, 1], 4, 16, 64)  # already longer than the table


def test_bad_table_entries_negative_lengths_and_empty_batches():
    _run(np.arange(0, 300, 7), np.ones(43), 24, 16, 90, bad=True, seed=3)
    _run([-5, 7, 3], [2, -1, 1], 4, 16, 9)
    _run([], [], 4, 16, 8)
    _run([], [], 4, 16, 8, pad=3)
    _run([3, 4], [0, 0], 4, 16, 8)


def test_out_is_written_and_checked():
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    out = nv.KVPlan(z(3), z(2), z(2), z(2, torch.int64), z(1), z(1))
    free = torch.arange(4, dtype=torch.int32, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    table = z((2, 4)).view(2, 4)
    r = nv.kv_plan(z(2), one, table, free, one[:1] * 4, page_size=8, num_pages=4, tokens=2, out=out)
    assert r is out and out.slots.tolist() == [24, 16] and table[:, 0].tolist() == [3, 2]
    with pytest.raises(ValueError):
        nv.kv_plan(z(2), one, table, free, one[:1], page_size=8, num_pages=5, tokens=2)
    with pytest.raises(TypeError):
        nv.kv_plan(z(2).long(), one, table, free, one[:1], page_size=8, num_pages=4, tokens=2)
    with pytest.raises(ValueError):
        nv.kv_plan(z(2), one, table[:1], free, one[:1], page_size=8, num_pages=4, tokens=2)
