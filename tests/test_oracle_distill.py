"""The float64 oracles of the distillation and processing calls: worked values, statuses, and
gradients against differences of the oracle's own forward pass."""
import numpy as np
import pytest

from oracle import distill as D
from oracle import processing as P


def all_of(n):
    return np.ones(n, bool)


def test_worked_divergences():
    p = np.array([0.4, 0.3, 0.2, 0.1])
    ids, q = np.array([1, 0]), np.array([0.5, 0.25])
    row = D.distill_row(np.log(p), ids, np.log(q), "forward", 2, 1.0, all_of(4))
    want = 0.5 * np.log(0.5 / 0.3) + 0.25 * np.log(0.25 / 0.4) + 0.25 * np.log(0.25 / 0.3)
    assert abs(row["loss"] - want) < 1e-15 and abs(row["logprob"] - np.log(0.2)) < 1e-15
    assert abs(row["stats"][3] - 0.3) < 1e-15
    row = D.distill_row(np.log(p), ids, np.log(q), "reverse", -1, 1.0, all_of(4))
    want = 0.3 * np.log(0.3 / 0.5) + 0.4 * np.log(0.4 / 0.25) + 0.3 * np.log(0.3 / 0.25)
    assert abs(row["loss"] - want) < 1e-15
    row = D.distill_row(np.log(p), ids, np.log(q) + 7.0, "truncated", -1, 1.0, all_of(4))
    want = 2 / 3 * np.log(2 / 3 / 0.3) + 1 / 3 * np.log(1 / 3 / 0.4)
    assert abs(row["loss"] - want) < 1e-14


def test_rows_at_the_edge():
    x, one = np.array([1.0, 2.0, 0.5]), all_of(3)
    for kind in ("forward", "reverse", "truncated"):
        none = D.distill_row(x, np.array([-1, -1]), np.zeros(2), kind, -1, 1.0, one)
        assert abs(none["loss"]) < 1e-15 and not none["d"].any() or abs(none["d"]).max() < 1e-15
    # every token has a slot: no term outside, whatever the teacher's sum is
    lq = np.log([0.3, 0.3, 0.3])
    row = D.distill_row(x, np.array([0, 1, 2]), lq, "forward", -1, 1.0, one)
    lp = x - np.log(np.exp(x).sum())
    assert abs(row["loss"] - 0.3 * (lq - lp).sum()) < 1e-15 and row["stats"][0] == -np.inf
    # a teacher's token that is not legal
    row = D.distill_row(x, np.array([0]), np.log([0.5]), "forward", -1, 1.0, np.array([False, True, True]))
    assert row["loss"] == np.inf and not row["d"].any()
    row = D.distill_row(x, np.array([0]), np.array([-np.inf]), "reverse", -1, 1.0, one)
    assert row["loss"] == np.inf and not row["d"].any()


def test_statuses():
    x, one, q = np.zeros(3), all_of(3), np.log([0.2, 0.2])
    f = lambda x=x, ids=(0, 1), q=q, kind="forward", t=-1, T=1.0, legal=one: D.distill_row(  # noqa: E731
        np.asarray(x, float), np.array(ids), np.asarray(q, float), kind, t, T, legal)["status"]
    assert f() == D.OK
    for bad in (dict(ids=(0, 3)), dict(ids=(-2, 0)), dict(ids=(1, 1)), dict(t=3), dict(t=-2), dict(T=0.0),
                dict(T=np.nan), dict(T=np.inf), dict(q=(0.1, -3.0))):
        assert f(**bad) == D.INVALID, bad
    assert f(q=(0.1, -3.0), kind="truncated") == D.OK
    assert f(q=(np.nan, -1.0)) == f(q=(np.inf, -1.0)) == f(q=(np.inf, -1.0), kind="truncated") == f(x=(0, 0, np.inf)) == D.NONFINITE
    assert f(legal=~one) == f(x=(-np.inf,) * 3) == D.EMPTY
    assert f(ids=(-1, 0), q=(np.nan, -1.0)) == D.OK  # unused slots are not looked at


@pytest.mark.parametrize("kind", ["forward", "reverse", "truncated"])
@pytest.mark.parametrize("V,K,T,masked", [(5, 2, 1.0, False), (17, 6, 0.7, True), (40, 12, 1.9, True), (6, 6, 0.8, False)])
def test_gradient_against_differences(kind, V, K, T, masked):
    rng = np.random.Generator(np.random.PCG64(V))
    x = rng.standard_normal(V) * 2
    legal = rng.random(V) < 0.6 if masked else all_of(V)
    ids = rng.permutation(np.nonzero(legal)[0])[:K]
    ids = np.concatenate([ids, np.full(K - len(ids), -1)])
    q = np.log(rng.dirichlet(np.ones(K + 1))[:K])
    t = int(np.nonzero(legal)[0][1])
    g, gl = 0.9, -0.4
    ok = D.distill_row(x, ids, q, kind, t, T, legal)
    d = D.grad_row(ok, ids, t, T, g, gl)

    def f(y):
        r = D.distill_row(y, ids, q, kind, t, T, legal)
        return g * r["loss"] + gl * r["logprob"]

    h = 1e-5  # truncation ~ h^2 = 1e-10, rounding ~ 1e-15 / h = 1e-10
    for j in range(V):
        e = np.zeros(V)
        e[j] = h
        assert abs((f(x + e) - f(x - e)) / (2 * h) - d[j]) < 2e-9, j
    # the slots' derivatives are the gradient's, by the scaled logit
    used = ids >= 0
    without = D.grad_row(ok, ids, -1, T, 1.0, 0.0)
    assert np.allclose(without[ids[used]] * T, ok["slot_grads"][used], atol=1e-14)


def test_processing():
    x = np.array([2.0, -1.0, 0.5, -np.inf, 3.0, 1.0])
    h = np.array([0, 1, 4, 4, -1, 3, 9, 4])
    st, v, _ = P.process_row(x, h, 3, 2.0, 0.25, 0.5, np.array([2, -1, 2, 5, 3]), np.array([1.0, np.nan, 0.5, -np.inf, 9.0]),
                             np.array([1, 1, 1, 1, 1, 1], bool))
    assert st == P.OK
    # 0 and 1 are the prompt's; 4 is both, and generated twice; 3 is -inf and stays
    assert list(v) == [1.0, -2.0, 2.0, -np.inf, 1.5 - 1.0 - 0.25, -np.inf]
    st, v, _ = P.process_row(x, h, 0, 2.0, 0.25, 0.5, np.zeros(0, int), np.zeros(0), np.arange(6) % 2 == 0)
    assert st == P.OK and list(v) == [1.0 - 0.75, -np.inf, 0.5, -np.inf, 1.5 - 1.5 - 0.25, -np.inf]
    for bad in (dict(theta=0.0), dict(theta=np.nan), dict(theta=np.inf), dict(presence=np.inf), dict(frequency=np.nan),
                dict(prompt=9), dict(prompt=-1), dict(bias=np.array([np.nan])), dict(bias=np.array([np.inf]))):
        a = dict(history=h, prompt=0, theta=1.5, presence=0.0, frequency=0.0, bias_ids=np.array([0]), bias=np.zeros(1)) | bad
        st, v, _ = P.process_row(x, a["history"], a["prompt"], a["theta"], a["presence"], a["frequency"], a["bias_ids"],
                                 a["bias"], np.zeros(6, bool))
        assert st == P.INVALID and np.array_equal(v, x), bad
