"""Pins of the dense operators' oracle: closed forms and hand-worked rows."""
import math

import numpy as np
import pytest

from oracle import dense


def test_quantise_closed_forms():
    p = np.array([[127.0, -63.5, 0.5, 1.5, 2.5, 0.0, -127.0, 64.0]])
    codes, scales = dense.quantise(p, 1.0, 0)
    assert codes.tolist() == [[127, -64, 0, 2, 2, 0, -127, 64]]      # ties to even
    assert scales.tolist() == [[1.0]]
    codes, scales = dense.quantise(np.zeros((1, 4)), 1.0, 0)
    assert not codes.any() and scales[0, 0] == 0
    codes, scales = dense.quantise(np.array([[1.0, np.inf, 2.0, 4.0]]), 1.0, 2)
    assert codes.tolist() == [[0, 0, 64, 127]] and np.isnan(scales[0, 0]) and scales[0, 1] == 4 / 127


def test_norm_closed_form_and_group_scales():
    x = np.full((1, 64), 3.0, dtype=np.float32)
    z, norm, codes, scales = dense.norm_q8(x, x, np.full(64, 2.0, np.float32), 0.0, 32)
    assert (z == 6).all() and np.allclose(norm, 2.0) and (codes == 127).all() and np.allclose(scales, 2.0 / 127)
    rs = np.random.default_rng(0)
    x = rs.standard_normal((3, 64)).astype(np.float32)
    _, norm, codes, scales = dense.norm_q8(x, None, None, 1e-6, 32)
    assert np.allclose(np.sqrt((norm ** 2).mean(-1)), 1.0, atol=1e-5)
    back = codes.reshape(3, 2, 32) * scales[..., None]
    assert np.abs(back.reshape(3, 64) - norm).max() <= scales.max() / 2 * (1 + 1e-12)


def test_a_row_that_is_not_finite_has_nan_scales():
    x = np.ones((2, 32), dtype=np.float32)
    x[1, 5] = np.nan
    _, norm, codes, scales = dense.norm_q8(x, None, None, 1e-6, 0)
    assert np.isfinite(scales[0]).all() and np.isnan(scales[1]).all() and not codes[1].any() and np.isnan(norm[1]).all()


def test_linear_by_hand():
    a, w = np.array([[1.0, 2.0]]), np.array([[3.0, 4.0], [-1.0, 0.5]])
    out, pre, mag = dense.linear(a, w, bias=[1.0, 0.0], residual=[[10.0, 20.0]])
    assert out.tolist() == [[22.0, 20.0]] and mag.tolist() == [[11.0, 2.0]]
    out, _, _ = dense.linear(a, w, a_scale=[2.0], w_scale=[0.5, 3.0])
    assert out.tolist() == [[11.0, 0.0]]


def test_activations():
    v = np.array([-2.0, 0.0, 1.0])
    assert dense.act(v, "relu").tolist() == [0, 0, 1]
    assert np.allclose(dense.act(v, "silu"), [-2 / (1 + math.exp(2)), 0, 1 / (1 + math.exp(-1))])
    assert np.allclose(dense.act(v, "gelu"), [-0.04550026389635842, 0, 0.8413447460685429])


L4 = np.log(np.array([0.1, 0.4, 0.2, 0.3]))


@pytest.mark.parametrize("kw,want", [
    (dict(u=0.0), (0, 0.1)), (dict(u=0.05), (0, 0.1)), (dict(u=0.15), (1, 0.4)), (dict(u=0.55), (2, 0.2)),
    (dict(u=0.99), (3, 0.3)), (dict(u=0.5, top_k=1), (1, 1.0)), (dict(u=0.9, top_k=2), (3, 3 / 7)),
    (dict(u=0.0, top_p=0.65), (1, 4 / 7)), (dict(u=0.99, top_p=0.75), (3, 3 / 9)), (dict(u=0.5, top_p=0.0), (1, 1.0)),
    (dict(u=0.0, min_p=0.6), (1, 4 / 7)), (dict(u=0.3, temperature=0), (1, 1.0)),
    # top-k first, then the prefix of what is left: of (0.4, 0.3) half is reached by the first alone
    (dict(u=0.9, top_k=2, top_p=0.5), (1, 1.0)),
])
def test_sampling_by_hand(kw, want):
    i, p = dense.sample_row(L4, **kw)
    assert i == want[0] and abs(p - want[1]) < 1e-12


def test_sampling_ties_masks_and_infinities():
    assert dense.sample_row([1.0, 1.0, 1.0], top_k=2, u=0.99) == (1, 0.5)          # ties keep the lower indices
    assert dense.sample_row([-np.inf, 2.0, np.nan], u=0.0) == (1, 1.0)
    assert dense.sample_row([-np.inf, np.nan], u=0.5) == (-1, 0.0)
    assert dense.sample_row([np.inf, 3.0, np.inf], u=0.7) == (2, 0.5)
    low = np.finfo(np.float32).min
    assert dense.sample_row([low, low], u=0.6) == (1, 0.5)
    assert dense.sample_row([0.0, -100.0], u=1 - 2.0 ** -24) == (0, 1.0)           # below 2^-64 there is no weight
