"""CPU pins of the 64-bit statement of the int8 routed experts
(oracle/experts.py) against closed forms, exact rational arithmetic and
brute force."""
import itertools
from fractions import Fraction

import numpy as np
import pytest

from oracle import experts as ox


def test_route_hand_worked():
    a = np.array([[0.0, np.log(3.0), np.log(2.0), -np.inf]])
    ids, w = ox.route(a, 2)
    assert ids.tolist() == [[1, 2]]
    assert np.allclose(w, [[0.6, 0.4]])
    ids, w = ox.route(a, 2, renormalize=False, scale=6.0)
    assert np.allclose(w, [[3.0, 2.0]])
    # a bias changes the choice, not the weights
    ids, w = ox.route(a, 2, bias=[1.0, 0.0, 0.0, 5.0], renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1 / 6, 1 / 2]])
    # nothing to choose
    ids, w = ox.route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[-1, -1]] and not w.any()


def test_route_ties_and_groups():
    ids, _ = ox.route(np.zeros((1, 8)), 3)
    assert ids.tolist() == [[0, 1, 2]]
    a = np.array([[9.0, 0, 0, 0, 8, 8, 0, 0]])
    # without a bias the group of the 9 and that of the 8s stay, each by its best
    assert ox.route(a, 3, n_groups=4, topk_groups=2)[0].tolist() == [[0, 4, 5]]
    # with one, groups go by the sum of their two best
    s = 1 / (1 + np.exp(-a[0]))
    ids, _ = ox.route(a, 2, bias=np.zeros(8), n_groups=4, topk_groups=1, score="sigmoid")
    assert s[4] + s[5] > s[0] + s[1] and ids.tolist() == [[4, 5]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_against_full_enumeration(score, with_bias):
    rng = np.random.default_rng(3)
    a = rng.normal(size=(20, 6))
    b = rng.normal(size=6) if with_bias else None
    p = np.exp(a) / np.exp(a).sum(1)[:, None] if score == "softmax" else 1 / (1 + np.exp(-a))
    v = p + (0 if b is None else b)
    ids, w = ox.route(a, 3, bias=b, score=score, renormalize=False)
    for i in range(len(a)):
        best = max(itertools.combinations(range(6), 3), key=lambda c: sum(v[i, list(c)]))
        assert sorted(ids[i]) == list(best)
        assert np.allclose(w[i], p[i, ids[i]])


def test_quantize_against_fractions():
    rng = np.random.default_rng(5)
    z = np.round(rng.normal(size=(12, 32)) * 64) / 64  # few bits: many exact halves
    q, scale = ox.int8_quantize(z)
    for i in range(len(z)):
        amax = max(abs(Fraction(float(v))) for v in z[i])
        for j in range(z.shape[1]):
            assert round(127 * Fraction(float(z[i, j])) / amax) == q[i, j]  # halves to even
        assert scale[i] == pytest.approx(float(amax / 127), rel=1e-15)


def test_quantize_special_rows():
    z = np.array([[0.0, -0.0], [1.0, np.inf], [np.nan, 1.0], [-3.0, 1.5]])
    q, scale = ox.int8_quantize(z)
    assert q[:3].tolist() == [[0, 0]] * 3 and q[3].tolist() == [-127, 64]  # 63.5 goes to 64
    assert scale[0] == 0 and np.isnan(scale[1:3]).all()


def test_experts_reduce_to_one_dense_expert():
    rng = np.random.default_rng(7)
    m, hidden, inter = 3, 32, 16
    xq, xs = rng.integers(-127, 128, (m, hidden)), rng.uniform(0.01, 0.02, m)
    w13, s13 = rng.integers(-127, 128, (2, 2 * inter, hidden)), rng.uniform(1e-3, 2e-3, (2, 2 * inter))
    w2, s2 = rng.integers(-127, 128, (2, hidden, inter)), rng.uniform(1e-3, 2e-3, (2, hidden))
    ids = np.array([[1, -1], [1, 1], [5, -1]])
    g = np.array([[0.5, 0.7], [0.25, 0.5], [1.0, 1.0]])
    y, bound = ox.experts_int8(xq, xs, w13, s13, w2, s2, ids, g)
    x = xq * xs[:, None]
    h = x @ (w13[1] * s13[1][:, None]).T
    act = h[:, :inter] / (1 + np.exp(-h[:, :inter])) * h[:, inter:]
    dense = act @ (w2[1] * s2[1][:, None]).T
    # int8 activations: half a step of the row in each of inter products
    step = np.abs(act).max(1)[:, None] / 254 * np.abs(w2[1] * s2[1][:, None]).sum(1)
    assert np.all(np.abs(y[0] - 0.5 * dense[0]) <= 0.5 * step[0])
    assert np.all(np.abs(y[1] - 0.75 * dense[1]) <= 0.75 * step[1])
    assert not y[2].any() and np.all(bound >= 0)
