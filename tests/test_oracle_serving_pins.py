"""The fp64 oracle of the gated delta rule, the RMS norm and the log probabilities against cases
worked by hand and, where there is one, another formula of the same thing."""
import numpy as np

from oracle import serving


def test_delta_rule_by_hand():
    # one head of two keys and two values; S [value, key]
    q, k = np.zeros((1, 2, 1, 2)), np.zeros((1, 2, 1, 2))
    v = np.zeros((1, 2, 1, 2))
    k[0, 0, 0], k[0, 1, 0] = (1, 0), (0, 1)
    q[0, :, 0] = (1, 2)
    v[0, 0, 0], v[0, 1, 0] = (3, 5), (7, 9)
    a, b = np.log(np.full((1, 2, 1), 0.5)), np.full((1, 2, 1), 0.5)
    S = np.array([[[[2.0, 4.0], [6.0, 8.0]]]])
    out = serving.gated_delta(q, k, v, a, b, S, scale=1.0, l2=False)[0]
    # t = 0: S = [[1, 2], [3, 4]]; u = 0.5 ((3, 5) - (1, 3)) = (1, 1); S = [[2, 2], [4, 4]]; o = (6, 12)
    # t = 1: S = [[1, 1], [2, 2]]; u = 0.5 ((7, 9) - (1, 2)) = (3, 3.5); S = [[1, 4], [2, 5.5]]; o = (9, 13)
    np.testing.assert_allclose(out[0, :, 0], [[6, 12], [9, 13]], rtol=1e-14)
    np.testing.assert_allclose(S[0, 0], [[1, 4], [2, 5.5]], rtol=1e-14)


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0, 1.0, 1.0, 1.0, 1.0]])
    # the mean squares are 6.25 and 1, beside an epsilon of 1e-6
    y, left = serving.rms_norm(x, np.full(4, 2.0), group=4)
    np.testing.assert_allclose(y, [[2.4, 3.2, 0, 0, 2, 2, 2, 2]], rtol=1e-6)
    y, left = serving.rms_norm(x, np.full(8, 1.0), residual=x, unit=True)
    np.testing.assert_allclose(left, 2 * x)
    np.testing.assert_allclose(y, 4 * x / np.sqrt(4 * 29 / 8), rtol=1e-6)


def test_log_probabilities_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.125, 0.125]])) + 3.0
    lp, ent, ids, best = serving.token_logprobs(x[None], np.array([[1]]), 3)
    np.testing.assert_allclose(lp, [[np.log(0.25)]], rtol=1e-14)
    np.testing.assert_allclose(ent, [[1.75 * np.log(2.0)]], rtol=1e-14)
    assert ids.tolist() == [[[0, 1, 2]]]
    np.testing.assert_allclose(best, np.log([[[0.5, 0.25, 0.125]]]), rtol=1e-14)
