"""Attention over the paged NVFP4 cache where its numbers' range counts:
weights far below the largest one, unusable amaxes, infinite queries."""
import numpy as np
import pytest

import kv_reference as R
from helpers import dev_bf16
from test_gpu_kv_attention import SG, _dev_cache, _make, _queries, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
nv = pytest.importorskip("nvfp4_block_scaled_02_amd")


@pytest.mark.parametrize("form", ["few rows", "few rows in pieces", "many rows"])
@pytest.mark.parametrize("gap", [8.0, 14.0, 16.0, 17.0, 17.5, 18.0, 20.0])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_large_score_over_a_long_flat_tail(d, gap, form):
    """A first key whose score is `gap` above all others and whose value is 0:
    what comes out is the tail's, n exp(-gap) / (1 + n exp(-gap))."""
    n = 6000 if form == "many rows" else 20000
    new = 70 if form == "many rows" else 1
    max_len = 128 if form == "few rows" else n  # the bound of a launch that cuts no keys
    c = _make([n], 64, 1, d, 31, garbage=False)
    c["amax"] = [np.array([6 * SG], np.float32)] * 2  # outer scales of 1
    c["kc"][:], c["ks"][:] = 0, 0x38
    vc, vs = np.full_like(c["kc"], 0x22), c["ks"].copy()  # values of 1
    p = c["table"][0, 0]
    c["kc"][p, 0, 0, 0] = 0x07  # (6, 0, ..)
    vc[p, 0, 0] = 0
    c["vc"], c["vs"] = R.pages_of(vc), R.pages_of(vs)
    q = np.zeros((new, 2, d))
    q[:, :, 0] = gap
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    out, lse = nv.kv_attention(dev_bf16(R.bits(q)), _dev_cache(c), torch.from_numpy(c["table"]).cuda(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"), cu, scale=1 / 6, want_lse=True,
                               max_seq_len=max_len)
    tail = (n - new + np.arange(new)) * np.exp(-gap)  # keys after the first, up to the query's own
    want, want_lse = tail / (1 + tail), gap + np.log1p(tail)
    # a weight rounds to binary16: 2^-11 of it, and below 2^-21 of the largest
    # one 2^-32 of that; the exponent's argument is good to a few 2^-24 of it;
    # the sums are of binary32, and the output rounds once
    rel = R.FP16 + 8 * gap * R.F32 + (n + 64) * R.F32
    mass = rel * tail + n * 2.0 ** -32
    tol = R.BF16 * want + 2 * (mass + rel * want) + R.F32
    o = out.float().cpu().numpy().astype(np.float64)
    assert (np.abs(o - want[:, None, None]) <= tol[:, None, None]).all(), float((np.abs(o - want[:, None, None]) / want[:, None, None]).max())
    l = lse.cpu().numpy().astype(np.float64)
    tol = (mass + rel) / (1 + tail) + 4 * R.F32 * np.abs(want_lse)
    assert (np.abs(l - want_lse[:, None]) <= tol[:, None]).all()


@pytest.mark.parametrize("amax", [np.nan, np.inf, -1.0])
@pytest.mark.parametrize("lens,new", [([2, 9], [4, 3]), ([50, 40], [130, 33])])
def test_rows_that_attend_nothing_under_an_unusable_amax(lens, new, amax):
    """A key amax that is no amax makes NaN of the rows that attend a key, and
    of no others: queries before the first token still give 0 and -inf."""
    c = _make(lens, 8, 2, 64, 32)
    c["amax"][0][0] = amax
    o, l = _run(c, _queries(sum(new), 4, 64, 32), lens, new)
    none = new[0] - lens[0]
    assert (o[:none] == 0).all() and np.isneginf(l[:none]).all()
    assert np.isnan(o[none:, :2]).all() and np.isfinite(o[none:, 2:]).all()


@pytest.mark.parametrize("lens,new", [([1, 5, 40, 40], [1, 1, 1, 2]), ([150], [140])])
@pytest.mark.parametrize("x", [0x7F80, 0xFF80])
def test_infinite_queries_against_keys_of_one_sign(lens, new, x):
    """exp(-inf + inf) is no number: a row whose scores are all infinite is NaN
    whatever their sign, unlike a row that attends nothing."""
    c = _make(lens, 16, 1, 128, 33)
    used = c["ks"][..., :1] != 0x7F
    c["kc"][..., :1] = np.where(used, (c["kc"][..., :1] & 0xF0) | 3, c["kc"][..., :1])  # value 0: +1.5 everywhere
    qb = _queries(sum(new), 2, 128, 33)
    qb[:, 0, 0] = x
    for scale in (0.1, -0.1):
        o, l = _run(c, qb, lens, new, scale=scale)
        assert np.isnan(o[:, 0]).all() and np.isnan(l[:, 0]).all()
        assert np.isfinite(o[:, 1]).all() and np.isfinite(l[:, 1]).all()
