"""Pins of the oracle's 4-bit cache, rotary positions and token probabilities:
worked cases, and properties that the formulas have by themselves."""

import numpy as np
import pytest

import oracle

S = oracle.serving


def test_codes4_worked():
    x = np.zeros((1, 64))
    x[0, :16] = np.arange(16)                        # 0 .. 15: steps of 1
    codes, scale, offset = S.codes4(x)
    assert float(scale[0]) == 1.0 and float(offset[0]) == -64.0
    # byte 4 g + i: channel 8 g + i low, 8 g + i + 4 high
    assert codes[0, :8].tolist() == [0x40, 0x51, 0x62, 0x73, 0xc8, 0xd9, 0xea, 0xfb]
    assert np.array_equal(S.values4(codes, scale, offset), x)


def test_codes4_edges():
    flat = np.full((1, 64), 3.25)
    codes, scale, offset = S.codes4(flat)
    assert float(scale[0]) == 0.0 and not codes.any() and np.array_equal(S.values4(codes, scale, offset), flat)
    far = np.zeros((1, 64))
    far[0, 0], far[0, 1] = np.inf, -np.inf
    codes, scale, offset = S.codes4(far)
    v = S.values4(codes, scale, offset)
    assert np.isfinite(v).all() and abs(v[0, 0] - 4096) < 40 and abs(v[0, 1] + 4096) < 40
    far[0, 2] = np.nan
    codes, scale, offset = S.codes4(far)
    assert np.isnan(S.values4(codes, scale, offset)).all() and not codes.any()


def test_codes4_error_is_half_a_step():
    x = np.random.default_rng(0).normal(size=(200, 128))
    codes, scale, offset = S.codes4(x)
    s = scale.astype(np.float64)[:, None]
    # half a step; the ends by what scale and offset are rounded (79 scales and an
    # offset, 2^-11 of each); the value's own rounding to fp16
    slack = (79 * s + np.abs(offset.astype(np.float64))[:, None]) * 2.0 ** -11 + np.abs(x) * 2.0 ** -11
    assert np.all(np.abs(S.values4(codes, scale, offset) - x) <= s / 2 + slack)


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotary_properties(neighbours):
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(16) / 16)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    at = lambda x, p: S.rotary(x, np.array([p]), f, 1.0, neighbours)  # noqa: E731
    assert np.allclose(at(q, 0), q) and np.array_equal(at(q, 7)[..., 32:], q[..., 32:])
    # a score depends on the distance alone, and lengths stay
    assert np.allclose((at(q, 90) * at(k, 73)).sum(), (at(q, 1017) * at(k, 1000)).sum())
    assert np.allclose((at(q, 90) ** 2).sum(), (q ** 2).sum())
    one = np.zeros((1, 1, 64))
    one[..., 0] = 1.0
    assert np.allclose(at(one, 1)[0, 0, [0, 1 if neighbours else 16]], [np.cos(1), np.sin(1)])


def test_token_probs_worked():
    logits = np.log(np.array([[1.0, 2.0, 4.0, 8.0], [1.0, 2.0, 4.0, 8.0]]))
    args = ([3], [0, 1], 4, [[1, 1]], None, [1], [[]], [None, None])
    p = S.token_probs(logits, [[1.0, 1.0, 0.0, 0.0]], *args)
    assert np.allclose(p[0], np.array([1, 2, 4, 8]) / 15) and np.allclose(p[1], p[0])
    # token 1 twice in the history, once in the prompt: one counts; the draft counts from the next row on
    p = S.token_probs(logits, [[1.0, 1.0, 0.0, np.log(2)]], *args)
    assert np.allclose(p[0], np.array([1, 1, 4, 8]) / 14) and np.allclose(p[1], np.array([1, 1, 4, 4]) / 10)
    p = S.token_probs(logits, [[0.5, 1.0, 0.0, 0.0]], *args)
    assert np.allclose(p[0], np.array([1, 4, 16, 64]) / 85)
    # repeats: positive logits are divided, others multiplied
    p = S.token_probs(logits, [[1.0, 2.0, 0.0, 0.0]], *args)
    assert np.allclose(p[0], np.array([1, 2 ** 0.5, 4, 8]) / (13 + 2 ** 0.5))
    p = S.token_probs(logits - 10, [[0.0, 2.0, 0.0, 0.0]], *args)
    assert p[0].tolist() == [0, 0, 0, 1] and p[1].tolist() == [0, 0, 1, 0]
    none = np.zeros(4, bool)
    p = S.token_probs(logits, [[1.0, 1.0, 0.0, 0.0]], [3], [0, 1], 4, [[]], None, [0], [[(2, -np.inf), (2, np.log(2))]],
                      [none, None])
    assert not p[0].any() and np.allclose(p[1], np.array([1, 2, 8, 8]) / 19)
