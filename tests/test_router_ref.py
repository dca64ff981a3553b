"""The 64-bit reference of the scored router against itself: the gradient against
central differences, the choice against a sort by hand, the masked cases."""
import numpy as np
import pytest

import router_ref as R


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(3)
    for _ in range(10):
        l = 2 * rng.standard_normal(12)
        idx = R.choose(l, 4, score)
        dw = rng.standard_normal(4)
        got, _ = R.backward(dw, l, idx, score, renormalise, 2.5)
        h = 1e-6
        for e in range(12):
            up, down = l.copy(), l.copy()
            up[e] += h
            down[e] -= h
            # differences carry h^2 and 1e-16 / h: 1e-10 each, times weights of a few units
            want = (dw @ (R.weights(up, idx, score, renormalise, 2.5)
                          - R.weights(down, idx, score, renormalise, 2.5))) / (2 * h)
            assert abs(got[e] - want) < 1e-8


def test_groups_by_hand():
    l = np.array([5., 0., 4., 4., 9., -9., 1., 1.])
    # ranks by two: 5, 8, 0, 2; by one: 5, 4, 9, 1 (by logits: no balance)
    assert R.choose(l, 3, "sigmoid", 4, 2, 1).tolist() == [4, 0, 1]
    s, _ = R.scores(l, "sigmoid")
    two = s.reshape(4, 2).sum(1)
    kept = np.argsort(-two, kind="stable")[:2]
    got = R.choose(l, 3, "sigmoid", 4, 2, 2)
    assert set(got // 2) <= set(kept)


def test_masked_rows():
    inf = np.inf
    assert R.choose(np.array([-inf, 1., np.nan, 0.]), 3).tolist() == [1, 3, 0]
    assert R.choose(np.full(4, -inf), 2).tolist() == [0, 1]
    assert R.weights(np.full(4, -inf), np.array([0, 1])).tolist() == [0., 0.]
    w = R.weights(np.array([inf, 0., inf]), np.array([0, 2]))
    assert w.tolist() == [0.5, 0.5]
    w = R.weights(np.array([-800., -801.]), np.array([0, 1]), "sigmoid")
    assert abs(w[0] - 1 / (1 + np.exp(-1))) < 1e-15
