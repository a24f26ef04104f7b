"""Whose memory the key/value-cache calls use."""
import threading

import pytest

from helpers import dev_bf16
from test_gpu_kv_attention import _dev_cache, _make, _queries

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")


def _split_call(seed=41):
    """Arguments of an attention call whose keys are cut into pieces."""
    lens = [3000, 20]
    c = _make(lens, 16, 2, 128, seed)
    return (dev_bf16(_queries(2, 8, 128, seed)), _dev_cache(c), torch.from_numpy(c["table"]).cuda(),
            torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _struct(launch):
    return launch._args[0]._obj


def test_prepared_attentions_have_buffers_of_their_own():
    args = _split_call()
    want = nv.kv_attention(*args)  # the stream's own buffers exist
    launches = [nv.prepare(nv.kv_attention, *args) for _ in range(2)]
    for field in ("workspace", "counters"):
        own = [getattr(_struct(l), field) for l, _ in launches]
        shared = [t.data_ptr() for t in (*nv.kv._ATTENTION_WORKSPACES.values(), *nv.kv._COUNTERS.values())]
        assert None not in own and own[0] != own[1] and not set(own) & set(shared), field
    for launch, out in launches:
        out.zero_()
        for _ in range(3):
            launch()
        assert torch.equal(out, want)


def test_prepared_gradients_have_buffers_of_their_own():
    x = torch.randn(50, 4, 64, device="cuda").bfloat16()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    want = nv.qk_norm_rope_bwd(x, x, x, x, q_weight=w, k_weight=w)
    launches = [nv.prepare(nv.qk_norm_rope_bwd, x, x, x, x, q_weight=w, k_weight=w) for _ in range(2)]
    own = [l._args[-1] for l, _ in launches]
    assert own[0] != own[1] and not set(own) & {t.data_ptr() for t in nv.kv._BWD_WORKSPACES.values()}
    for launch, got in launches:
        for _ in range(3):
            launch()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_threads_on_one_stream_do_not_mix_their_pieces(monkeypatch):
    """A call may be two launches with one workspace between them: no other
    thread's call on that stream may come between."""
    args = _split_call(42)
    nv.kv_attention(*args)
    inside, entered, both = threading.Lock(), [], threading.Event()
    real = nv.kv._invoke

    def invoke(entry, *rest):
        with inside:
            entered.append(threading.get_ident())
            if len(entered) > 1:
                both.set()
        alone = not both.wait(0.5) if entered[0] == threading.get_ident() else True
        real(entry, *rest)
        if not alone:
            entered.append("mixed")

    monkeypatch.setattr(nv.kv, "_invoke", invoke)
    threads = [threading.Thread(target=nv.kv_attention, args=args) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(entered) == 2 and len(set(entered)) == 2


def test_a_cache_cannot_be_given_other_memory():
    """The calls pass the addresses that the cache was made with."""
    cache = _split_call(43)[1]
    for field, value in (("k_codes", cache.k_codes.clone()), ("v_amax", cache.v_amax.clone()),
                         ("global_max", 448.0), ("num_pages", 1)):
        with pytest.raises(AttributeError):
            setattr(cache, field, value)
    assert cache == cache and cache != _split_call(43)[1]


def test_plan_outputs_may_not_be_its_inputs():
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    ctx, new, table = z(2), z(2) + 1, z(8).view(2, 4)
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), z(1) + 4
    kw = dict(page_size=8, num_pages=4, tokens=2)

    def out(**other):
        return nv.KVPlan(**{**dict(cu_new=z(3), seq_lens=z(2), positions=z(2), slots=z(2, torch.int64),
                                   free_count=z(1), refused=z(1)), **other})

    lens = torch.cat([ctx, new])
    for o, c in ((out(seq_lens=ctx), ctx), (out(seq_lens=new), ctx), (out(free_count=count), ctx),
                 (out(refused=free[3:]), ctx), (out(positions=table.view(-1)[3:5]), ctx),
                 (out(seq_lens=lens[1:3]), lens[:2]), (out(slots=lens.view(torch.int64)), lens[:2])):
        with pytest.raises(ValueError, match="share memory"):
            nv.kv_plan(c, new, table, free, count, **kw, out=o)
    # beside each other in one allocation
    o = out(seq_lens=lens[2:])
    assert nv.kv_plan(lens[:2], new, table, free, count, **kw, out=o).seq_lens.tolist() == [1, 1]
