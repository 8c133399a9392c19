"""Pins of the float64 oracle of the operators around headwise QK-Norm (CPU):
closed forms, brute force and differences."""

import math

import numpy as np
import pytest

from oracle import operators as O


def test_rotation_closed_forms():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = (np.zeros((1, 4)), np.ones((1, 4)))      # 90 degrees: (a, b) -> (-b, a)
    assert O.rotate(x, *quarter, False).reshape(-1).tolist() == [-5, -6, -7, -8, 1, 2, 3, 4]
    assert O.rotate(x, *quarter, True).reshape(-1).tolist() == [-2, 1, -4, 3, -6, 5, -8, 7]
    half = (np.zeros((1, 2)), np.ones((1, 2)))         # only the first four columns
    assert O.rotate(x, *half, False).reshape(-1).tolist() == [-3, -4, 1, 2, 5, 6, 7, 8]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_turns_back(interleaved):
    r = np.random.default_rng(3)
    x, a = r.normal(size=(5, 3, 16)), r.normal(size=(5, 6))
    y = O.rotate(x, np.cos(a), np.sin(a), interleaved)
    np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
    np.testing.assert_allclose(O.rotate(y, np.cos(a), np.sin(a), interleaved, back=True), x, atol=1e-14)
    assert np.array_equal(y[..., 12:], x[..., 12:])


def test_rotated_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(4)
    q, k, f = r.normal(size=(1, 1, 32)), r.normal(size=(1, 1, 32)), r.uniform(0.01, 1, size=16)

    def score(i, j):
        a, b = (i * f)[None], (j * f)[None]
        return float((O.rotate(q, np.cos(a), np.sin(a), False) * O.rotate(k, np.cos(b), np.sin(b), False)).sum())

    assert math.isclose(score(7, 3), score(104, 100), rel_tol=1e-12)


@pytest.mark.parametrize("stride,interleaved,rot", [(0, False, 8), (8, True, 8), (10, False, 4), (0, True, 0)])
def test_gradients_against_differences(stride, interleaved, rot):
    r = np.random.default_rng(5)
    T, heads, d = 3, 4, 8
    x, dy = r.normal(size=(T, heads * d)), r.normal(size=(T, heads * d))
    gamma = r.normal(1, 0.2, size=(heads - 1) * stride + d)
    ang = r.normal(size=(T, rot // 2))
    cos, sin = (np.cos(ang), np.sin(ang)) if rot else (None, None)

    def loss(x, gamma):
        return float((O.norm_rope(x, gamma, 1e-6, d, stride, cos, sin, interleaved).reshape(T, -1) * dy).sum())

    dx, dgamma, _, _ = O.norm_rope_backward(x, dy, gamma, 1e-6, d, stride, cos, sin, interleaved)
    h = 1e-6
    for i in range(T):
        for j in range(heads * d):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((loss(x + e, gamma) - loss(x - e, gamma)) / (2 * h) - dx.reshape(T, -1)[i, j]) < 1e-7
    for j in range(gamma.size):
        e = np.zeros_like(gamma)
        e[j] = h
        assert abs((loss(x, gamma + e) - loss(x, gamma - e)) / (2 * h) - dgamma[j]) < 1e-7


def test_mxfp4_by_hand():
    x = np.zeros(32)
    x[:8] = [6, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, 5]   # largest 6: E = 0; every border is a tie
    codes, scale, value = O.mxfp4_quantize(x)
    assert scale.tolist() == [127]
    assert value[:8].tolist() == [6, 0, 1, -1, 2, 2, 4, 4]
    assert codes[:4].tolist() == [7 | 0 << 4, 2 | (2 | 8) << 4, 4 | 4 << 4, 6 | 6 << 4]
    assert O.mxfp4_quantize(x * 2.0 ** 7)[1].tolist() == [134]
    # saturation: 7.9 is nearest to 6, the largest
    x[0] = 7.9
    assert O.mxfp4_quantize(x)[2][0] == 6
    # zero block, tiny block, huge block
    assert O.mxfp4_quantize(np.zeros(32))[1].tolist() == [27]
    assert O.mxfp4_quantize(np.full(32, 2.0 ** -120))[2].tolist() == [0.0] * 32
    assert O.mxfp4_quantize(np.full(32, 3.0e38))[1].tolist() == [252]
    x[3] = np.nan
    assert O.mxfp4_quantize(x)[1].tolist() == [255] and np.isnan(O.mxfp4_quantize(x)[2]).all()


def test_mxfp4_is_nearest_by_brute_force():
    r = np.random.default_rng(6)
    x = r.normal(size=(40, 64)) * np.exp(r.normal(size=(40, 1)) * 5)
    codes, scale, value = O.mxfp4_quantize(x)
    assert np.array_equal(O.mxfp4_values(codes, scale), value)
    grid = np.concatenate((O.E2M1, -O.E2M1))
    for i in range(40):
        for blk in range(2):
            b = x[i, 32 * blk:32 * blk + 32]
            E = math.floor(math.log2(np.abs(b).max())) - 2
            assert scale[i, blk] == E + 127
            for j, v in enumerate(b):
                best = min(abs(v - g * 2.0 ** E) for g in grid)
                assert abs(v - value[i, 32 * blk + j]) == best


def test_attention_closed_forms():
    r = np.random.default_rng(7)
    K, V = np.zeros((6, 2, 4)), r.normal(size=(6, 2, 4))
    q = r.normal(size=(3, 4, 4))
    out, _, some = O.attend(q, K, V, 3, 0.5, True, 0)      # equal scores: plain means
    for i in range(3):
        for h in range(4):
            np.testing.assert_allclose(out[i, h], V[:4 + i, h // 2].mean(0), atol=1e-15)
    assert some.all()
    out, _, _ = O.attend(q, K, V, 3, 0.5, True, 1)         # a window of one: the token itself
    np.testing.assert_allclose(out[2, 3], V[5, 1])
    out, _, _ = O.attend(q, K, V, 3, 0.5, False, 0)
    np.testing.assert_allclose(out[0, 0], V[:, 0].mean(0))
    out, _, some = O.attend(r.normal(size=(3, 4, 4)), K[:2], V[:2], 3, 0.5, True, 0)   # more queries than tokens
    assert some.tolist() == [False, True, True] and not out[0].any()
