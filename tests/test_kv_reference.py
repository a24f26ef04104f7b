"""The tests' own plain implementations: gradients against differences, the
layouts against their descriptions, attention against a direct sum."""
import math

import numpy as np
import pytest

import kv_reference as R


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("weight", [True, False])
def test_gradient_against_differences(pairs, weight):
    rng = np.random.default_rng(0)
    t, h, d, rot = 2, 2, 64, 32
    x, pos = rng.standard_normal((t, h, d)), np.array([3, 9])
    w = 1 + 0.2 * rng.standard_normal(d) if weight else None
    a = np.arange(20)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    cos, sin = np.cos(a), np.sin(a)
    gy = rng.standard_normal((t, h, d))
    dx, dw, _, _ = R.norm_rope_bwd(gy, x, w, pos, cos, sin, 1e-6, pairs)
    f = lambda x, w: (R.norm_rope(x, w, pos, cos, sin, 1e-6, pairs)[0] * gy).sum()  # noqa: E731
    for _ in range(12):
        i = tuple(rng.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = 1e-6
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-6 - dx[i]) < 1e-7
        if weight:
            e = np.zeros(d)
            e[i[2]] = 1e-6
            assert abs((f(x, w + e) - f(x, w - e)) / 2e-6 - dw[i[2]]) < 1e-7


def test_layouts():
    rng = np.random.default_rng(1)
    v = rng.integers(0, 256, (3, 2, 16, 32), dtype=np.uint8)
    p = R.pages_of(v)
    assert p.shape == (3, 2, 2, 32, 8) and p[1, 1, 1, 7, 3] == v[1, 1, 11, 7]
    assert np.array_equal(R.rows_of(p), v)
    codes = np.array([[0x21] + [0] * 7 + [0x9F] + [0] * 7], np.uint8)
    rows = R.decode_rows(codes, np.array([[0x38, 0x40]], np.uint8))  # scales 1 and 2
    assert rows[0, 0] == 0.5 and rows[0, 1] == 1.0 and rows[0, 16] == -12.0 and rows[0, 17] == -1.0


def test_attention_of_two_keys():
    d, sg = 64, 256.0
    kc, ks = np.zeros((1, 1, 8, 32), np.uint8), np.full((1, 1, 8, 4), 0x38, np.uint8)
    kc[0, 0, 1, 0] = 0x02  # key 1 = (1, 0, ..)
    vc = np.zeros((1, 1, 8, 32), np.uint8)
    vc[0, 0, 0, 0], vc[0, 0, 1, 0] = 0x04, 0x06  # values 2 and 4
    amax = np.array([6 * sg], np.float32)  # alpha = 1
    q = np.zeros((1, 1, d))
    q[0, 0, 0] = 3.0
    o, lse, tol, _ = R.attention(q, kc, ks, R.pages_of(vc), R.pages_of(ks), amax, amax, sg,
                                 np.zeros((1, 1), np.int64), [2], [0, 1], 8, 0.5, True, 0)
    e = math.exp(1.5)
    assert abs(o[0, 0, 0] - (2 + 4 * e) / (1 + e)) < 1e-12 and abs(lse[0, 0] - math.log(1 + e)) < 1e-12
    assert 0 < tol[0, 0, 0] < 0.1
