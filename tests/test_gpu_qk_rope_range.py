"""Norm and rotation's gradient at the ends of its range: no eps, and rows whose
squares leave binary32.  The tolerances are those of test_gpu_qk_rope.py."""
import numpy as np
import pytest

import kv_reference as R
from helpers import dev_bf16, dev_f32
from test_gpu_qk_rope import _bits_of, _bwd_close, _inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")


def _gradient(x, w, pos, cos, sin, eps, seed):
    """The gradients of both sides beside the formula's."""
    rng = np.random.default_rng(seed)
    g = [R.bits(rng.standard_normal(v.shape)) for v in x]
    got = nv.qk_norm_rope_bwd(dev_bf16(g[0]), dev_bf16(g[1]), dev_bf16(x[0]), dev_bf16(x[1]),
                              torch.from_numpy(pos).cuda(), dev_f32(cos), dev_f32(sin),
                              q_weight=dev_bf16(w[0]), k_weight=dev_bf16(w[1]), eps=eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        want = [R.norm_rope_bwd(R.f64(g[i]), R.f64(x[i]), R.f64(w[i]), pos, cos, sin, eps, "halves")
                for i in range(2)]
    return got, want


def _weights_close(got, dw, wmag, d, what):
    tol = (12 + np.log2(d)) * R.F32 * wmag + R.F32 * np.abs(dw)
    assert (np.abs(got.cpu().numpy().astype(np.float64) - dw) <= tol).all(), what


@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("t,hq,hk", [(1, 1, 2), (5, 7, 1), (300, 12, 3)])
def test_no_eps_and_spare_head_places(t, hq, hk, d):
    """Head counts that leave places of a wavefront without a head: those add
    nothing to the weights' gradients, whatever 0^-1/2 is."""
    x, w, pos, cos, sin = _inputs(t, hq, hk, d, d if d % 64 == 0 else 32, t + d)
    got, want = _gradient(x, w, pos, cos, sin, 0.0, t)
    for i, (dx, dw, mag, wmag) in enumerate(want):
        _bwd_close(_bits_of(got[i]), dx, mag, d, ("dx", i))
        _weights_close(got[2 + i], dw, wmag, d, ("dw", i))


def test_no_eps_and_a_row_of_zeros():
    """0 * 0^-1/2 is no number: in its own row, and in the sums over rows."""
    x, w, pos, cos, sin = _inputs(4, 3, 1, 64, 64, 9)
    x[0][2, 1] = 0
    got, want = _gradient(x, w, pos, cos, sin, 0.0, 9)
    bad = np.zeros((4, 3), bool)
    bad[2, 1] = True
    dq = _bits_of(got[0])
    assert np.isnan(R.f64(dq)[bad]).all()
    _bwd_close(dq[~bad], want[0][0][~bad], want[0][2][~bad], 64, "the other rows")
    assert torch.isnan(got[2]).all()
    _weights_close(got[3], want[1][1], want[1][3], 64, "the keys' side")


@pytest.mark.parametrize("d,hq,hk", [(64, 3, 2), (128, 4, 1), (192, 2, 3), (256, 5, 2)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_whose_squares_leave_binary32(d, hq, hk, eps):
    """The forward call norms rows of any size, and so does its gradient:
    magnitudes from 2^-110 to 2^110 beside ordinary ones."""
    t = 40
    x, w, pos, cos, sin = _inputs(t, hq, hk, d, d, d)
    rng = np.random.default_rng(d)
    for i in range(2):
        e = rng.choice([-110, -70, -58, 0, 0, 45, 58, 70, 110], (t, x[i].shape[1], 1))
        x[i] = R.bits(rng.standard_normal(x[i].shape) * 2.0 ** e)
    got, want = _gradient(x, w, pos, cos, sin, eps, d)
    for i, (dx, dw, mag, wmag) in enumerate(want):
        assert (np.abs(dx) < 3e38).all() and np.abs(dx).max(-1).min() > 0
        _bwd_close(_bits_of(got[i]), dx, mag, d, ("dx", i))
        _weights_close(got[2 + i], dw, wmag, d, ("dw", i))
