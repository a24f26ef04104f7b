"""Norm and rotation of query and key heads, and the gradient, against the
64-bit formula.  Forward: binary64 inside, so one rounding to bf16 (behind one
to binary32) and 2^-45 of the terms added.  Gradient: binary32 inside."""
import numpy as np
import pytest

import kv_reference as R
from helpers import dev_bf16, dev_f32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")

EPS = 1e-6


def _inputs(t, hq, hk, d, rot, seed, far=0):
    rng = np.random.default_rng(seed)
    x = [R.bits(rng.standard_normal((t, h, d)) * np.exp(rng.normal(0, 2, (t, h, 1)))) for h in (hq, hk)]
    w = [R.bits(1 + 0.3 * rng.standard_normal(d)) for _ in range(2)]
    top = 500 + far
    pos = rng.integers(far, top, t).astype(np.int32)
    f = 10000.0 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 2))
    a = np.arange(top)[:, None] * f
    return x, w, pos, np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _close(got_bits, ref, mag, what):
    got = R.f64(got_bits)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what
    tol = (R.BF16 + R.F32) * np.abs(ref) + 2.0 ** -45 * mag + 2.0 ** -134
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    ok = ~nan & ~inf
    assert (np.abs(got - ref)[ok] <= tol[ok]).all(), (what, np.abs(got - ref)[ok].max())


CASES = [  # tokens, q heads, k heads, D, rot
    (1, 1, 1, 128, 128), (1, 32, 8, 128, 128), (3, 7, 1, 64, 64), (17, 4, 2, 128, 64),
    (5, 3, 5, 96, 32), (9, 2, 2, 32, 32), (4, 6, 3, 192, 192), (130, 2, 1, 256, 128),
    (33, 5, 2, 160, 96), (2, 1, 3, 224, 0), (1, 64, 8, 64, 32),
]


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("t,hq,hk,d,rot", CASES)
def test_forward(t, hq, hk, d, rot, pairs):
    x, w, pos, cos, sin = _inputs(t, hq, hk, d, rot, t * d + rot, far=20000)
    tab = (torch.from_numpy(pos).cuda(), dev_f32(cos), dev_f32(sin)) if rot else (None,) * 3
    c, s = (cos, sin) if rot else (None, None)
    for qw, kw in ((True, True), (False, True), (True, False), (False, False)):
        q, k = nv.qk_norm_rope(dev_bf16(x[0]), dev_bf16(x[1]), *tab,
                               q_weight=dev_bf16(w[0]) if qw else None,
                               k_weight=dev_bf16(w[1]) if kw else None, eps=EPS, pairs=pairs)
        for got, xb, wb, n in ((q, x[0], w[0] if qw else None, "q"), (k, x[1], w[1] if kw else None, "k")):
            ref, mag = R.norm_rope(R.f64(xb), None if wb is None else R.f64(wb), pos, c, s, EPS, pairs)
            _close(_bits_of(got), ref, mag, (n, qw, kw))


def test_views_of_a_projection_in_place_and_one_side():
    x, w, pos, cos, sin = _inputs(21, 6, 2, 128, 128, 5)
    rng = np.random.default_rng(0)
    qkv = dev_bf16(np.concatenate([x[0], x[1], R.bits(rng.standard_normal((21, 2, 128)))], 1))
    keep = qkv.clone()
    tab = (torch.from_numpy(pos).cuda(), dev_f32(cos), dev_f32(sin))
    kw = dict(q_weight=dev_bf16(w[0]), k_weight=dev_bf16(w[1]))
    q, k = nv.qk_norm_rope(qkv[:, :6], qkv[:, 6:8], *tab, **kw)
    assert torch.equal(qkv, keep)
    only, none = nv.qk_norm_rope(qkv[:, :6], None, *tab, q_weight=kw["q_weight"])
    assert none is None and torch.equal(only, q)
    none, only = nv.qk_norm_rope(None, qkv[:, 6:8], *tab, k_weight=kw["k_weight"])
    assert none is None and torch.equal(only, k)
    nv.qk_norm_rope(qkv[:, :6], qkv[:, 6:8], *tab, out=(qkv[:, :6], qkv[:, 6:8]), **kw)
    assert torch.equal(qkv[:, :6], q) and torch.equal(qkv[:, 6:8], k)
    assert torch.equal(qkv[:, 8:], keep[:, 8:])
    # one token of a wider buffer, other tokens' strides
    q1, k1 = nv.qk_norm_rope(keep[4:5, :6], keep[4:5, 6:8], tab[0][4:5], *tab[1:], **kw)
    assert torch.equal(q1[0], q[4]) and torch.equal(k1[0], k[4])
    q2, k2 = nv.qk_norm_rope(keep[::2, :6], keep[::2, 6:8], tab[0][::2].contiguous(), *tab[1:], **kw)
    assert torch.equal(q2, q[::2]) and torch.equal(k2, k[::2])


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_special_rows_stay_in_their_row(pairs):
    x, w, pos, cos, sin = _inputs(6, 2, 1, 64, 64, 8)
    x[0][1, 0, 5] = 0x7F80          # an infinity
    x[0][2, 1, 7] = 0x7FC0          # a NaN
    x[0][3] = 0                     # zeros: 0 * eps^-1/2
    x[0][4] = 0x0001                # the smallest subnormal
    pos[5], pos[0] = len(cos), -1   # outside the table
    q, _ = nv.qk_norm_rope(dev_bf16(x[0]), dev_bf16(x[1]), torch.from_numpy(pos).cuda(), dev_f32(cos),
                           dev_f32(sin), q_weight=dev_bf16(w[0]), k_weight=dev_bf16(w[1]), pairs=pairs)
    with np.errstate(invalid="ignore"):
        ref, mag = R.norm_rope(R.f64(x[0]), R.f64(w[0]), pos, cos, sin, EPS, pairs)
    got = R.f64(_bits_of(q))
    assert np.isnan(got[[0, 5]]).all() and np.isnan(got[2, 1]).all()
    assert np.isnan(got[1, 0]).any() and np.isfinite(got[1, 1]).all() and np.isfinite(got[2, 0]).all()
    assert (got[3] == 0).all()
    ok = np.array([[False, False], [False, True], [True, False], [True, True], [True, True], [False, False]])
    _close(_bits_of(q)[ok], ref[ok], mag[ok], "finite rows")


# ------------------------------------------------------------------ gradient
def _bwd_close(got, ref, mag, d, what):
    # binary32: each of about 3 log2(D) + 12 roundings moves a term by 2^-24
    tol = R.BF16 * np.abs(ref) + (3 * np.log2(d) + 12) * R.F32 * mag
    assert (np.abs(R.f64(got) - ref) <= tol).all(), (what, np.abs(R.f64(got) - ref).max())


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("t,hq,hk,d,rot", CASES + [(700, 9, 2, 64, 64), (2100, 4, 4, 128, 128)])
def test_gradient(t, hq, hk, d, rot, pairs):
    x, w, pos, cos, sin = _inputs(t, hq, hk, d, rot, t * d + rot + 1)
    rng = np.random.default_rng(t)
    g = [R.bits(rng.standard_normal((t, h, d))) for h in (hq, hk)]
    tab = (torch.from_numpy(pos).cuda(), dev_f32(cos), dev_f32(sin)) if rot else (None,) * 3
    c, s = (cos, sin) if rot else (None, None)
    for qw, kw in ((True, True), (False, True), (False, False)):
        r = nv.qk_norm_rope_bwd(dev_bf16(g[0]), dev_bf16(g[1]), dev_bf16(x[0]), dev_bf16(x[1]), *tab,
                                q_weight=dev_bf16(w[0]) if qw else None,
                                k_weight=dev_bf16(w[1]) if kw else None, eps=EPS, pairs=pairs)
        for i, has in ((0, qw), (1, kw)):
            dx, dw, mag, wmag = R.norm_rope_bwd(R.f64(g[i]), R.f64(x[i]), R.f64(w[i]) if has else None,
                                                pos, c, s, EPS, pairs)
            _bwd_close(_bits_of(r[i]), dx, mag, d, ("dx", i, qw, kw))
            if not has:
                assert r[2 + i] is None
                continue
            # each term within 12 + log2(D) binary32 roundings, the sum in binary64
            tol = (12 + np.log2(d)) * R.F32 * wmag + R.F32 * np.abs(dw)
            assert (np.abs(r[2 + i].cpu().numpy().astype(np.float64) - dw) <= tol).all(), ("dw", i)


def test_gradient_repeats_bit_for_bit_and_takes_views():
    t, hq, hk, d = 3000, 8, 2, 128
    x, w, pos, cos, sin = _inputs(t, hq, hk, d, d, 3)
    rng = np.random.default_rng(1)
    qkv = dev_bf16(np.concatenate(x, 1))
    g = dev_bf16(R.bits(rng.standard_normal((t, hq + hk, d))))
    tab = (torch.from_numpy(pos).cuda(), dev_f32(cos), dev_f32(sin))
    kw = dict(q_weight=dev_bf16(w[0]), k_weight=dev_bf16(w[1]))
    first = nv.qk_norm_rope_bwd(g[:, :hq], g[:, hq:], qkv[:, :hq], qkv[:, hq:], *tab, **kw)
    dense = nv.qk_norm_rope_bwd(g[:, :hq].contiguous(), g[:, hq:].contiguous(), qkv[:, :hq].contiguous(),
                                qkv[:, hq:].contiguous(), *tab, **kw)
    dqkv = torch.zeros_like(qkv)
    into = nv.qk_norm_rope_bwd(g[:, :hq], g[:, hq:], qkv[:, :hq], qkv[:, hq:], *tab,
                               out={"dq": dqkv[:, :hq], "dk": dqkv[:, hq:]}, **kw)
    for r in (dense, into):
        for a, b in zip(first, r):
            assert torch.equal(a, b)
    # the queries' side alone adds the same terms (its sums may split otherwise)
    alone = nv.qk_norm_rope_bwd(g[:, :hq], None, qkv[:, :hq], None, *tab, q_weight=kw["q_weight"])
    assert torch.equal(alone[0], first[0]) and alone[1] is None and alone[3] is None


def test_gradient_without_tokens_is_zero():
    z = lambda h: torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = nv.qk_norm_rope_bwd(z(2), z(1), z(2), z(1), q_weight=w, k_weight=w,
                            out={"dq_weight": torch.full((64,), 7.0, device="cuda")})
    assert r[0].shape == (0, 2, 64) and (r[2] == 0).all() and (r[3] == 0).all()
    q, k = nv.qk_norm_rope(z(2), z(1), q_weight=w, k_weight=w)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)


def test_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    cos = torch.ones(8, 32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: nv.qk_norm_rope(x.float(), x), lambda: nv.qk_norm_rope(x, x, q_weight=w.float()),
                lambda: nv.qk_norm_rope(x, x, pos.long(), cos, cos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: nv.qk_norm_rope(x, x[:3]), lambda: nv.qk_norm_rope(x, x[..., :32]),
                lambda: nv.qk_norm_rope(x.transpose(1, 2), x), lambda: nv.qk_norm_rope(x, x, pos, cos, None),
                lambda: nv.qk_norm_rope(x, x, pos[:3], cos, cos), lambda: nv.qk_norm_rope(x, x, pos, cos, cos[:7]),
                lambda: nv.qk_norm_rope(x, x, q_weight=w[:32]), lambda: nv.qk_norm_rope(x[:, 0], x),
                lambda: nv.qk_norm_rope(x[:, ::2], x[:, ::2].expand(4, 2, 64)),
                lambda: nv.qk_norm_rope(x[:1].expand(4, 2, 64), x), lambda: nv.qk_norm_rope(x, None, k_weight=w),
                lambda: nv.qk_norm_rope_bwd(x, None, x, x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nv._native.NativeError):
        nv.qk_norm_rope(x, x, eps=-1.0)
