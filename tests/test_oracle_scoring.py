"""The float64 scoring oracle: worked values, and its gradient against
differences of its own forward pass."""
import numpy as np
import pytest

from oracle import scoring as S


def test_worked_example():
    p = np.array([0.4, 0.3, 0.2, 0.1])
    r = S.score_row(np.log(p), 2, 1.0, np.ones(4, bool), 3)
    assert abs(r["logprob"] - np.log(0.2)) < 1e-15 and r["rank"] == 2
    assert abs(r["entropy"] + (p * np.log(p)).sum()) < 1e-15
    assert list(r["top_ids"]) == [0, 1, 2] and np.allclose(r["top_logprobs"], np.log(p[:3]))
    r = S.score_row(np.log(p), 2, 1.0, np.array([0, 0, 1, 1], bool), 3)
    assert abs(r["logprob"] - np.log(2 / 3)) < 1e-15 and r["rank"] == 0
    assert list(r["top_ids"]) == [2, 3, -1] and r["top_logprobs"][2] == -np.inf
    r = S.score_row(np.log(p), 0, 1.0, np.array([0, 0, 1, 1], bool), 0)
    assert r["logprob"] == -np.inf and r["rank"] == 2 and r["status"] == S.OK


def test_temperature_and_ties():
    r = S.score_row(np.array([1.0, 3.0, 3.0, 2.0]), 2, 0.5, np.ones(4, bool), 4)
    assert list(r["top_ids"]) == [1, 2, 3, 0] and r["rank"] == 1
    w = np.exp(np.array([-4.0, 0, 0, -2.0]))
    assert abs(r["logprob"] + np.log(w.sum())) < 1e-15
    assert r["stats"] == (3.0, pytest.approx(np.log(w.sum()), abs=1e-15))


def test_statuses():
    one, inf, nan = np.ones(2, bool), np.inf, np.nan
    assert S.score_row(np.array([1.0, inf]), 0, 1.0, one, 0)["status"] == S.NONFINITE
    assert S.score_row(np.array([1.0, nan]), 0, 1.0, np.array([1, 0], bool), 0)["status"] == S.OK
    assert S.score_row(np.array([-inf, -inf]), 0, 1.0, one, 0)["status"] == S.EMPTY
    for T in (0.0, -1.0, nan, inf):
        assert S.score_row(np.array([1.0, 2.0]), 0, T, one, 0)["status"] == S.INVALID
    for t in (-2, 2):
        assert S.score_row(np.array([1.0, 2.0]), t, 1.0, one, 0)["status"] == S.INVALID


@pytest.mark.parametrize("V,T,masked", [(5, 1.0, False), (17, 0.7, True), (40, 1.9, True)])
def test_gradient_against_differences(V, T, masked):
    rng = np.random.Generator(np.random.PCG64(V))
    x = rng.standard_normal(V) * 2
    legal = rng.random(V) < 0.6 if masked else np.ones(V, bool)
    t = int(np.nonzero(legal)[0][0])
    g, gh = -0.7, 0.3

    def f(y):
        r = S.score_row(y, t, T, legal, 0)
        return g * r["logprob"] + gh * r["entropy"]

    d = S.grad_row(S.score_row(x, t, T, legal, 0), t, T, g, gh)
    h = 1e-5  # truncation ~ h^2 = 1e-10, rounding ~ 1e-15 / h = 1e-10
    for j in range(V):
        e = np.zeros(V)
        e[j] = h
        assert abs((f(x + e) - f(x - e)) / (2 * h) - d[j]) < 2e-9, j
