"""Worked cases for the serving operators' oracle."""

import math

import numpy as np

from oracle import serving


def test_block_norm_by_hand():
    y = np.zeros((2, 1, 128))
    y[0, 0, :] = 1.0
    y[1, 0, :] = 2.0                      # u = 3 everywhere, rms 3
    resid = np.full((1, 128), 0.5)
    gate = np.full((1, 128), 4.0)
    h, z = serving.block_norm(y, resid, np.full(128, 2.0), np.full(128, 3.0), gate, 1, 0.25, 0.0, False, False)
    assert np.allclose(h, 0.5 + 0.25 * 4.0 * 2.0)
    assert np.allclose(z, 3.0)            # a constant row normed is 1
    # the transform of a constant block is its sum / sqrt(128) in place 0
    _, z = serving.block_norm(y, resid, None, np.ones(128), None, 1, 1.0, 0.0, False, True)
    assert np.allclose(z[0, 0], math.sqrt(128.0)) and np.allclose(z[0, 1:], 0.0)


def test_attention_by_hand():
    # one head of two channels; positions 0..2 on pages 5, 5, 3 of two positions each
    k = np.zeros((6, 1, 2, 2))
    v = np.zeros((6, 1, 2, 2))
    k[5, 0, 0], k[5, 0, 1], k[3, 0, 0] = [math.log(2.0), 0], [0, 0], [math.log(3.0), 7]
    v[5, 0, :, 0], v[5, 0, :, 1], v[3, 0, :, 0] = [1, 2], [4, 8], [100, 200]
    q = np.array([[[1.0, 0.0]], [[1.0, 0.0]]])
    table = np.array([[5, 3]])
    out, lse, mean, _ = serving.paged_attention(q, k, v, table, [0, 2], [3], 1.0, 0)
    assert np.allclose(out[0, 0], [(2 * 1 + 4) / 3, (2 * 2 + 8) / 3])   # weights 2, 1
    assert np.allclose(lse[:, 0], [math.log(3.0), math.log(6.0)])      # and 2, 1, 3
    assert np.allclose(out[1, 0], [(2 + 4 + 300) / 6, (4 + 8 + 600) / 6]) and np.allclose(mean, out)
    out, lse, _, _ = serving.paged_attention(q, k, v, table, [0, 2], [3], 1.0, 1)
    assert np.allclose(out[:, 0], [[4, 8], [100, 200]])                # a window of one: itself
    # more tokens than positions: the first ones see nothing
    out, lse, _, _ = serving.paged_attention(q, k, v, table, [0, 2], [1], 1.0, 0)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and np.allclose(out[1, 0], [1, 2])
    # a page that is not there
    out, _, _, _ = serving.paged_attention(q, k, v, np.array([[9, 3]]), [0, 2], [3], 1.0, 0)
    assert np.all(out[0] == 0) and np.allclose(out[1, 0], [100, 200])


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25], [0.25, 0.5, 0.25], [0.125, 0.125, 0.75], [0.0, 1.0, 0.0]])
    q = np.array([[0.25, 0.5, 0.25], [0.0, 0.25, 0.75]])
    cu = [0, 2, 2]
    # token 0 (p 0.5, q 0.25) is kept at any u; token 2 (p 0.25, q 0.75) while u < 1/3
    acc, tok = serving.verify_draft(p, q, [0, 2], [0.99, 0.5], [0.4, 0.3], cu, 2)
    # not kept: p - q = (.25, .25, -) -> total .5, goal .2: token 0; sequence 1 draws from p[3]
    assert acc.tolist() == [1, 0] and tok.tolist() == [[0, 0, -1], [1, -1, -1]]
    acc, tok = serving.verify_draft(p, q, [0, 2], [0.99, 0.25], [0.4, 0.3], cu, 2)
    assert acc.tolist() == [2, 0] and tok[0].tolist() == [0, 2, 2]
    # a certain drafter: kept while u < p, else p without the token
    acc, tok = serving.verify_draft(p, None, [0, 2], [0.5, 0.0], [0.5, 0.0], cu, 2)
    assert acc.tolist() == [0, 0] and tok[0].tolist() == [2, -1, -1]  # weights (0, .25, .25), goal .25: past it is token 2
    # an edge: u q = p is not kept; a draw of 0 takes the first weight that is not 0
    acc, tok = serving.verify_draft(p[:2], p[:1], [1], [1.0], [0.0], [0, 1], 1)
    assert acc.tolist() == [0] and tok[0].tolist() == [0, -1]  # p - q leaves nothing: p itself
