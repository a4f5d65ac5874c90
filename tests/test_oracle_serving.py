"""The serving operators' oracle against closed forms and differences (CPU)."""

import math

import numpy as np
import pytest

from oracle import formats as F
from oracle import serving as S


def test_rms_norm_closed_forms():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    y, h = S.rms_norm(x, np.array([2.0, 1.0]), 0.5)
    assert np.allclose(y[0], np.array([6.0, 4.0]) / math.sqrt(13.0), rtol=1e-15) and not y[1].any()
    y2, h2 = S.rms_norm(x - 1, np.array([2.0, 1.0]), 0.5, np.ones((2, 2)))
    assert np.array_equal(y2, y) and np.array_equal(h2, x)


@pytest.mark.parametrize("act,slope0", [("relu", None), ("gelu", 0.5), ("gelu_tanh", 0.5), ("silu", 0.5)])
def test_activations(act, slope0):
    z = np.array([[-1e3, 0.0, 1e3]])
    y = S.activation(z, act)
    assert np.allclose(y, [[0.0, 0.0, 1e3]], atol=1e-9)
    if slope0 is not None:
        d = (S.activation(np.array([[1e-6]]), act) - S.activation(np.array([[-1e-6]]), act)) / 2e-6
        assert abs(d[0, 0] - slope0) < 1e-6
    t = np.linspace(-6, 6, 4001)[None]
    assert np.abs(np.diff(S.activation(t, act)) / np.diff(t)).max() < 1.13  # the slope the tests count with


def test_swiglu_pairs_sixteen_columns():
    z = np.random.default_rng(0).standard_normal((2, 64))
    y = S.activation(z, "swiglu")
    for j in range(32):
        a = z[:, 32 * (j // 16) + j % 16]
        assert np.allclose(y[:, j], a / (1 + np.exp(-a)) * z[:, 32 * (j // 16) + 16 + j % 16], rtol=1e-14)


def test_cover_exponent():
    assert S.cover_exponent(0.0) == -127 and S.cover_exponent(448.0) == 0 and S.cover_exponent(448.0001) == 1
    assert S.cover_exponent(1e-45) == -127 and S.cover_exponent(3.4e38) == 120
    for a in np.random.default_rng(1).lognormal(0, 10, 1000):
        e = S.cover_exponent(a)
        assert a <= 448 * 2.0 ** e and a > 448 * 2.0 ** (e - 1)


def test_append_rounds_once_and_again_when_the_scale_grows():
    c = S.Cache(*(np.zeros((2, 1, 16, 2), np.uint8) for _ in range(2)), *(np.full((2, 1), 9) for _ in range(2)))
    c.append(np.full((3, 1, 2), 1.1), np.full((3, 1, 2), -2.0), [[1]], [3], [0, 3])
    assert c.ke[1, 0] == -8 and c.ve[1, 0] == -7  # the old exponent 9 of an unused block is dropped
    k = F.e4m3_decode(c.k[1, 0, :3]) * 2.0 ** -8
    assert (np.abs(k - 1.1) <= 2.0 ** -4 / 2 + 1e-12).all()
    c.append(np.full((1, 1, 2), 3e5), np.zeros((1, 1, 2)), [[1]], [4], [0, 1])
    assert c.ke[1, 0] == 10 and c.ve[1, 0] == -7
    assert (F.e4m3_decode(c.k[1, 0, :3]) == np.rint(k / 2.0 ** 10 * 512) / 512).all()  # below the normal range
    assert c.ke[0, 0] == 9


def test_attention_is_a_mean_under_equal_scores_and_picks_the_largest():
    rng = np.random.default_rng(3)
    v = F.e4m3_encode(rng.standard_normal((1, 1, 16, 2)).astype(np.float32))
    c = S.Cache(np.zeros((1, 1, 16, 2), np.uint8), v, np.zeros((1, 1), int), np.zeros((1, 1), int))
    out, lse, _, _ = S.attention(np.ones((3, 2, 2)), c, [[0]], [10], [0, 3], 1.0)
    w = F.e4m3_decode(v[0, 0])
    for i in range(3):
        assert np.allclose(out[i], w[:8 + i].mean(0)) and np.allclose(lse[i], math.log(8 + i))
    c.k[0, 0, 4] = 0x78  # 256
    out, _, _, _ = S.attention(np.ones((3, 2, 2)), c, [[0]], [10], [0, 3], 1.0)
    assert np.allclose(out, w[4])
    out, lse, _, _ = S.attention(np.ones((3, 2, 2)), c, [[5]], [10], [0, 3], 1.0)
    assert not out.any() and np.isneginf(lse).all()
    out, _, _, _ = S.attention(np.ones((3, 2, 2)), c, [[0]], [10], [0, 3], 1.0, window=1)
    assert np.allclose(out[:, 0], w[7:10])
