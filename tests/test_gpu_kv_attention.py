"""Attention over the paged NVFP4 cache against the definition in 64 bits;
the tolerance counts the roundings of the header's contract."""
import numpy as np
import pytest

import kv_reference as R
from helpers import dev_bf16, dev_f32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")

SG = 256.0


def _make(lens, page, h, d, seed, width=None, spare=3, garbage=True, spread=0.5):
    """A cache whose used tokens hold random codes and scales and whose other
    bytes are NaN scales and full codes; pages in random order."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    width = max(need + [1]) if width is None else width
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    used = np.zeros((pages, page), bool)
    at = 0
    for b, n in enumerate(lens):
        n = max(n, 0)
        m = min(need[b], width)
        table[b, :m] = order[at:at + m]
        for i in range(m):
            used[table[b, i], :max(0, min(page, n - i * page))] = True
        at += need[b]
    u = used[:, None, :, None]
    fill = lambda x, g: np.where(u, x, g if garbage else 0).astype(np.uint8)  # noqa: E731
    scale = lambda: np.clip(np.rint(0x38 + 8 * spread * rng.standard_normal((pages, h, page, d // 16))), 1, 0x7E)  # noqa: E731
    kc = fill(rng.integers(0, 256, (pages, h, page, d // 2)), 0xFF)
    vc = fill(rng.integers(0, 256, (pages, h, page, d // 2)), 0xFF)
    ks, vs = fill(scale(), 0x7F), fill(scale(), 0x7F)
    amax = [(6 * SG * rng.uniform(0.2, 0.5, h)).astype(np.float32) for _ in range(2)]
    return dict(kc=kc, ks=ks, vc=R.pages_of(vc), vs=R.pages_of(vs), amax=amax, table=table, page=page, h=h, d=d)


def _dev_cache(c):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return nv.KVCache(t(c["kc"]), t(c["ks"]), t(c["vc"]), t(c["vs"]), dev_f32(c["amax"][0]),
                      dev_f32(c["amax"][1]), SG)


def _queries(t, hq, d, seed, mult=1.0):
    rng = np.random.default_rng(seed + 99)
    return R.bits(mult * rng.standard_normal((t, hq, d)))


def _run(c, qb, lens, new, *, scale=None, causal=True, window=0, max_len=None, pad=0, q=None, what="", check=True):
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    one = all(n == 1 for n in new) and pad == 0
    q = dev_bf16(qb) if q is None else q
    cache = _dev_cache(c)
    args = (q, cache, torch.from_numpy(c["table"]).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kw = dict(scale=scale, causal=causal, window=window, max_seq_len=max_len, want_lse=True)
    out, lse = nv.kv_attention(*args, torch.from_numpy(cu).cuda(), **kw)
    if one:  # the form without cu_q is the same call
        out1, lse1 = nv.kv_attention(*args, None, **kw)
        assert torch.equal(out1.view(torch.int16), out.view(torch.int16)) and torch.equal(lse1.view(torch.int32), lse.view(torch.int32)), what
    again = nv.kv_attention(*args, torch.from_numpy(cu).cuda(), **{**kw, "want_lse": False})
    assert torch.equal(again.view(torch.int16), out.view(torch.int16)), "the same call twice"
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    if check:
        ro, rl, tol, toll = R.attention(R.f64(qb), c["kc"], c["ks"], c["vc"], c["vs"], *c["amax"], SG,
                                        c["table"].astype(np.int64), lens, cu, c["page"],
                                        c["d"] ** -0.5 if scale is None else scale, causal, window)
        nan = np.isnan(ro)
        assert np.array_equal(np.isnan(o), nan), (what, "NaN places")
        err = np.abs(o - ro)
        bad = ~nan & ~(err <= tol)
        assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.where(nan, 0, err / (tol + 1e-300)))))
        fin = np.isfinite(rl)
        assert np.array_equal(l[~fin], rl[~fin], equal_nan=True), (what, "lse")
        assert (np.abs(l[fin] - rl[fin]) <= toll[fin]).all(), (what, "lse")
    return o, l


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("hq,h", [(1, 1), (8, 2), (7, 1), (32, 8), (40, 2)])
def test_single_tokens(d, hq, h):
    lens = [1, 2, 31, 32, 33, 64, 100, 129, 257]
    c = _make(lens, 16, h, d, d + hq)
    _run(c, _queries(len(lens), hq, d, 1), lens, [1] * len(lens))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 256, 1024])
def test_pages(page):
    lens = [5, 8, 9, 63, 64, 65, 300, 1025]
    c = _make(lens, page, 2, 128, page)
    _run(c, _queries(len(lens), 8, 128, 2), lens, [1] * len(lens))


@pytest.mark.parametrize("new", [2, 3, 5, 8, 16, 17])
@pytest.mark.parametrize("d,hq,h", [(64, 4, 4), (128, 8, 2), (128, 14, 2), (256, 16, 1)])
def test_drafted_tokens(new, d, hq, h):
    lens = [new, new + 1, 40, 97, 300]
    c = _make(lens, 16, h, d, new)
    _run(c, _queries(new * len(lens), hq, d, new), lens, [new] * len(lens))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 7, 32, 100])
def test_prompts_behind_cached_tokens(causal, window):
    new, ctx = [130, 1, 0, 33, 70], [50, 90, 20, 0, 200]
    lens = [a + b for a, b in zip(new, ctx)]
    c = _make(lens, 32, 2, 64, 5)
    _run(c, _queries(sum(new), 6, 64, 5), lens, new, causal=causal, window=window)


@pytest.mark.parametrize("d,h,hq,page", [(128, 1, 4, 64), (256, 1, 2, 8), (192, 2, 4, 16), (64, 1, 1, 8)])
def test_longer_prompts(d, h, hq, page):
    new, ctx = [300, 129], [37, 0]
    lens = [a + b for a, b in zip(new, ctx)]
    c = _make(lens, page, h, d, d)
    _run(c, _queries(sum(new), hq, d, 6), lens, new)


def test_long_sequences_split():
    # few rows over a long axis: the work is split and joined
    lens = [20000, 7, 1, 12345]
    c = _make(lens, 64, 1, 128, 7)
    _run(c, _queries(4, 4, 128, 7), lens, [1] * 4)
    _run(c, _queries(4, 4, 128, 8), lens, [1] * 4, window=777)
    # the bound only sizes the launch: longer requests are computed in full
    _run(c, _queries(4, 4, 128, 9), lens, [1] * 4, max_len=128)
    _run(c, _queries(4, 4, 128, 9), lens, [1] * 4, max_len=0)
    new = [3, 1, 1, 4]
    _run(c, _queries(9, 4, 128, 10), lens, new)


def test_rows_that_attend_nothing():
    lens, new = [0, 2, 5, 0], [1, 4, 2, 3]  # empty requests, queries before the first token
    c = _make([8, 2, 5, 8], 8, 2, 128, 9)
    o, l = _run(c, _queries(10, 4, 128, 9), lens, new)
    for r in (0, 1, 2, 7, 8, 9):
        assert (o[r] == 0).all() and np.isneginf(l[r]).all()
    assert np.isfinite(l[3]).all()
    _run(c, _queries(4, 4, 128, 9), [0, -3, 5, 0], [1] * 4)


def test_padding_rows_are_zero():
    lens, new = [40, 9], [3, 2]
    c = _make(lens, 16, 2, 64, 10)
    qb = _queries(5 + 40, 4, 64, 10)
    o, l = _run(c, qb, lens, new, pad=40)
    assert (o[5:] == 0).all() and np.isneginf(l[5:]).all()


def test_bad_pages_are_not_attended():
    lens = [100, 100, 40]
    c = _make(lens, 16, 2, 128, 11)
    c["table"][0, 2], c["table"][1, 0], c["table"][1, 5] = -1, len(c["kc"]), 1 << 30
    c["table"][2, :] = -5  # nothing left
    o, l = _run(c, _queries(3, 4, 128, 11), lens, [1] * 3)
    assert (o[2] == 0).all()
    _run(c, _queries(60, 4, 128, 11), lens, [30, 20, 10])
    # longer than the table: what it names is attended
    c = _make([64, 64], 16, 1, 64, 12, width=4)
    _run(c, _queries(2, 2, 64, 12), [1000, 64], [1, 1])


def test_nan_keys_and_values_reach_the_rows_that_attend_them():
    lens, new = [90, 70], [60, 1]
    c = _make(lens, 16, 1, 128, 13)

    def at(b, j):
        return c["table"][b, j // 16], j % 16

    p, o = at(0, 50)
    c["ks"][p, 0, o, 3] = 0x7F          # a NaN key: rows from position 50 on
    p, o = at(0, 70)
    c["vs"][p, 0, o // 8, 2, o % 8] = 0x7F  # a NaN value block: 16 columns of rows from 70 on
    o_, _ = _run(c, _queries(61, 4, 128, 13), lens, new)
    assert np.isfinite(o_[:20]).all() and np.isnan(o_[20:60]).all() and np.isfinite(o_[60]).all()
    c["ks"][:] = np.where(c["ks"] == 0x7F, 0x30, c["ks"])
    o_, _ = _run(c, _queries(61, 4, 128, 13), lens, new)
    assert np.isfinite(o_[:40]).all() and np.isnan(o_[40:60, :, 32:48]).all()
    assert np.isfinite(o_[40:60, :, :32]).all() and np.isfinite(o_[40:60, :, 48:]).all()
    # behind a window the value is no longer seen
    o_, _ = _run(c, _queries(61, 4, 128, 13), lens, new, window=5)
    assert np.isnan(o_[40:45, :, 32:48]).all() and np.isfinite(o_[45:60]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_with_nan_and_bad_pages(d):
    """The same in the form for many rows: NaN keys and values, missing pages
    and garbage past the end, in tiles that rows attend in part."""
    lens, new = [210, 150], [180, 140]
    c = _make(lens, 16, 1, d, 20 + d)

    def at(b, j):
        return c["table"][b, j // 16], j % 16

    qb = _queries(320, 2, d, 20)
    p, o = at(0, 150)
    c["vs"][p, 0, o // 8, 1, o % 8] = 0x7F
    p, o = at(1, 60)
    c["ks"][p, 0, o, 2] = 0x7F
    o_, _ = _run(c, qb, lens, new)
    assert np.isfinite(o_[:120]).all() and np.isnan(o_[120:180, :, 16:32]).all()
    assert np.isfinite(o_[120:180, :, :16]).all() and np.isfinite(o_[180:230]).all() and np.isnan(o_[230:]).all()
    _run(c, qb, lens, new, window=20)
    _run(c, qb, lens, new, causal=False, window=33)
    c["table"][0, 3], c["table"][0, 9], c["table"][1, 1] = -1, 1 << 29, len(c["kc"])
    _run(c, qb, lens, new)
    _run(c, qb, [100, 150], new)  # rows before the first token
    c["table"][1, :] = -1
    o_, l = _run(c, qb, lens, new)
    assert (o_[180:] == 0).all() and np.isneginf(l[180:]).all()


def test_many_requests_and_uneven_rows():
    # more requests than one probe of 64 finds; prompts among single tokens
    rng = np.random.default_rng(21)
    new = rng.choice([0, 1, 1, 1, 3, 40], 300).tolist()
    lens = [n + int(k) for n, k in zip(new, rng.integers(0, 60, 300))]
    c = _make(lens, 8, 1, 64, 21)
    _run(c, _queries(sum(new), 2, 64, 21), lens, new)
    lens = rng.integers(0, 50, 700).tolist()
    c = _make(lens, 8, 1, 64, 22)
    _run(c, _queries(700, 2, 64, 22), lens, [1] * 700)


def test_special_queries():
    lens = [50] * 6
    c = _make(lens, 16, 1, 128, 14)
    qb = _queries(6, 4, 128, 14)
    qb[0, 0, 3], qb[1, 1, 4], qb[2] = 0x7FC0, 0x7F80, 0
    qb[3] = 0x0001                      # subnormals
    qb[4, :, ::2] = 0                   # a wide row: 2^40 next to small values
    qb[4, :, 7] = 0x5380
    o, l = _run(c, qb, lens, [1] * 6, scale=2.0 ** -40, check=False)
    assert np.isnan(o[0, 0]).all() and np.isfinite(o[0, 1:]).all()
    assert np.isnan(o[1, 1]).all() and np.isfinite(o[1, [0, 2, 3]]).all() and np.isfinite(o[2:]).all()
    qb[:2] = _queries(2, 4, 128, 15)
    _run(c, qb, lens, [1] * 6, scale=2.0 ** -40)
    _run(c, _queries(6, 4, 128, 14, mult=60.0), lens, [1] * 6)   # one-hot rows
    _run(c, _queries(6, 4, 128, 14, mult=1e-3), lens, [1] * 6)   # flat rows
    _run(c, _queries(6, 4, 128, 14), lens, [1] * 6, scale=-0.3)
    _run(c, _queries(6, 4, 128, 14), lens, [1] * 6, scale=0.0)


def test_extreme_scales_and_amaxes():
    lens = [70, 33]
    c = _make(lens, 16, 2, 64, 16)
    c["ks"][:, :, :, 0], c["vs"][:, :, :, 1] = 0x7E, 0x7E  # the largest block scale, 448
    c["ks"][:, :, :, 1], c["vs"][:, :, :, 0] = 0x01, 0x01  # the smallest
    _run(c, _queries(2, 4, 64, 16, mult=0.01), lens, [1, 1])
    _run(c, _queries(40, 4, 64, 16, mult=0.01), lens, [30, 10])
    c["amax"][0][0], c["amax"][1][1] = 0.0, 0.0  # alpha = 1
    _run(c, _queries(2, 4, 64, 16, mult=1e-4), lens, [1, 1])
    c["amax"][0][0] = np.nan
    o, _ = _run(c, _queries(2, 4, 64, 16, mult=1e-4), lens, [1, 1], check=False)
    assert np.isnan(o[:, :2]).all() and np.isfinite(o[:, 2:]).all()


def test_wide_head_groups():
    # more heads in a group than a tile has rows
    lens = [70, 3, 200]
    c = _make(lens, 16, 1, 128, 23)
    _run(c, _queries(3, 48, 128, 23), lens, [1] * 3)
    _run(c, _queries(3, 100, 128, 24), lens, [1] * 3)
    _run(c, _queries(8, 24, 128, 25), lens, [5, 1, 2])


def test_strided_queries_and_out():
    lens = [40, 100]
    c = _make(lens, 16, 2, 128, 17)
    qb = _queries(2, 12, 128, 17)
    wide = dev_bf16(qb)
    o, _ = _run(c, np.ascontiguousarray(qb[:, :8]), lens, [1, 1], q=wide[:, :8])
    cache, table = _dev_cache(c), torch.from_numpy(c["table"]).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert nv.kv_attention(wide[:, :8], cache, table, n, out=out) is out
    assert np.array_equal(out.float().cpu().numpy(), o)


def test_another_stream_and_prepared_launch():
    lens = [3000, 20]
    c = _make(lens, 16, 2, 128, 18)
    cache, table = _dev_cache(c), torch.from_numpy(c["table"]).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = dev_bf16(_queries(2, 8, 128, 18))
    want = nv.kv_attention(q, cache, table, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = nv.kv_attention(q, cache, table, n)
    launch, out = nv.prepare(nv.kv_attention, q, cache, table, n)
    launch()
    launch()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out, want)


def test_graph_of_a_decode_step():
    """Plan, append and attention captured once and replayed over changing
    lengths, with eager work between the replays, each against eager calls."""
    h, hq, d, page, batch, width = 2, 8, 128, 16, 5, 12
    pages = batch * width
    amax = torch.full((h,), 5.0, device="cuda")
    cos, sin = nv.rope_table(512, d)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    free = torch.randperm(pages, device="cuda").int()

    def fresh():
        return dict(cache=nv.kv_cache(pages, h, page, d, amax, amax), ctx=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                    table=torch.zeros(batch, width, dtype=torch.int32, device="cuda"),
                    count=torch.full((1,), pages, dtype=torch.int32, device="cuda"))

    qkv = torch.zeros(batch, hq + 2 * h, d, dtype=torch.bfloat16, device="cuda")
    new = torch.ones(batch, dtype=torch.int32, device="cuda")

    def step(s):
        p = nv.kv_plan(s["ctx"], new, s["table"], free, s["count"], page_size=page, num_pages=pages, tokens=batch)
        q = nv.kv_append(s["cache"], qkv[:, hq:hq + h], qkv[:, hq + h:], p.slots, q=qkv[:, :hq], positions=p.positions,
                         cos=cos, sin=sin, q_weight=w, k_weight=w)
        o = nv.kv_attention(q, s["cache"], s["table"], p.seq_lens)
        s["ctx"].copy_(p.seq_lens)
        s["count"].copy_(p.free_count)
        return o

    eager, graphed = fresh(), fresh()
    warm = fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(graphed)
    for i in range(40):
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        want = step(eager)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(eager["ctx"], graphed["ctx"]) and int(graphed["ctx"][0]) == i + 1
    for a in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(eager["cache"], a), getattr(graphed["cache"], a))


def test_refusals():
    one = torch.ones(2, device="cuda")
    cache = nv.kv_cache(4, 2, 16, 64, one, one)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: nv.kv_attention(q[..., :32], cache, table, lens), lambda: nv.kv_attention(q, cache, table[:2], lens),
                lambda: nv.kv_attention(q[:2], cache, table, lens), lambda: nv.kv_attention(q, cache, table, lens, cu[:3]),
                lambda: nv.kv_attention(q, cache, table, lens, out=q[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.kv_attention(q.float(), cache, table, lens), lambda: nv.kv_attention(q, cache, table.long(), lens),
                lambda: nv.kv_attention(q, cache, table, lens.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: nv.kv_attention(q[:, :3].contiguous(), cache, table, lens),
                lambda: nv.kv_attention(q, cache, table, lens, window=-1),
                lambda: nv.kv_attention(q, cache, table, lens, scale=float("nan")),
                lambda: nv.kv_attention(q, cache, table, lens, max_seq_len=-1)):
        with pytest.raises(nv._native.NativeError):
            bad()
    assert nv.kv_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 4, 64)


def test_window_past_every_position():
    """A window wider than any sequence attends as none does, to the last bit."""
    c = _make([700, 3, 90], 16, 2, 128, 71)
    qb = _queries(3 + 40, 8, 128, 71)
    for new in ([1, 1, 1], [40, 2, 1]):
        n = sum(new)
        runs = [_run(c, qb[:n], [700, 3, 90], new, window=w, check=w == 0) for w in (0, 2**31 - 1, 2**31, 2**63 - 1)]
        for o, l in runs[1:]:
            assert np.array_equal(o, runs[0][0]) and np.array_equal(l, runs[0][1])


@pytest.mark.parametrize("d,hq,h,lens,new", [
    (128, 32, 8, [8191], [1]), (128, 8, 2, [2000, 31, 700, 1999, 1], [1] * 5), (64, 4, 1, [5000], [1]),
    (192, 6, 2, [3000, 10], [1, 1]), (256, 4, 2, [4000, 0, 129], [1] * 3), (128, 8, 4, [6000, 300], [2, 1])])
def test_joined_in_the_first_launch_or_a_second(d, hq, h, lens, new):
    """With counters the pieces of a sequence are joined in the first launch,
    without (under capture) by a second one: the same bits, and the counters
    are left zero."""
    c = _make(lens, 16, h, d, 83)
    qb = _queries(sum(new), hq, d, 83)
    want, _ = _run(c, qb, lens, new)
    cache, q, table = _dev_cache(c), dev_bf16(qb), torch.from_numpy(c["table"]).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    counters = torch.zeros(nv.KV_COUNTER_BYTES, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        second = nv.kv_attention(q, cache, table, n, cu)
        first = nv.kv_attention(q, cache, table, n, cu, counters=counters)
    for _ in range(3):
        first.zero_(), second.zero_()
        g.replay()
        eager = nv.kv_attention(q, cache, table, n, cu, counters=counters)
        torch.cuda.synchronize()
        for o in (first, second, eager):
            assert np.array_equal(o.float().cpu().numpy().astype(np.float64), want)
        assert not counters.any()
