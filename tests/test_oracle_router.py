"""Pins of the routing oracle: rows worked out by hand, brute force over every
choice of k experts, and central differences of the weights."""

import itertools

import numpy as np
import pytest

from oracle import router


def test_rows_worked_out_by_hand():
    # logits 0 give sigmoid 1/2; ln 3 gives 3/4; -ln 3 gives 1/4
    l3 = np.log(3.0)
    x = np.array([[0.0, l3, -l3, l3]])
    idx, w = router.moe_route_topk(x, 3, score="sigmoid", renormalize=False)
    assert idx.tolist() == [[1, 3, 0]] and np.allclose(w, [[0.75, 0.75, 0.5]], atol=1e-15)
    idx, w = router.moe_route_topk(x, 2, score="sigmoid", scale=2.0)
    assert idx.tolist() == [[1, 3]] and np.allclose(w, [[1.0, 1.0]], atol=1e-15)
    # softmax of (0, ln 3, -ln 3, ln 3) = (3, 9, 1, 9) / 22
    idx, w = router.moe_route_topk(x, 3, score="softmax", renormalize=False)
    assert idx.tolist() == [[1, 3, 0]] and np.allclose(w, np.array([[9, 9, 3]]) / 22, atol=1e-15)
    idx, w = router.moe_route_topk(x, 3, score="softmax")
    assert np.allclose(w, np.array([[9, 9, 3]]) / 21, atol=1e-15)
    # a bias moves the choice and not the weights
    idx, w = router.moe_route_topk(x, 1, bias=[1.0, 0, 0, 0], score="sigmoid", renormalize=False)
    assert idx.tolist() == [[0]] and np.allclose(w, [[0.5]], atol=1e-15)


def test_groups_and_masks():
    ninf = -np.inf
    x = np.array([[3.0, -9.0, 2.0, 2.0, 1.0, 1.0]])
    # best single choice: group 0; best two together: group 1 (sigmoid)
    assert router.moe_route_topk(x, 1, score="sigmoid", n_group=3, group_top=1)[0].tolist() == [[0]]
    assert router.moe_route_topk(x, 2, score="sigmoid", n_group=3, group_top=2)[0].tolist() == [[2, 3]]
    # a group whose experts are all masked comes last, masked experts never
    x = np.array([[ninf, ninf, 2.0, ninf, 1.0, 1.0], [ninf] * 6])
    idx, w = router.moe_route_topk(x, 4, score="softmax", n_group=3, topk_group=2, group_top=2)
    assert idx.tolist() == [[2, 4, 5, -1], [-1] * 4]
    assert w[0, 3] == 0 and np.all(w[1] == 0) and abs(w[0].sum() - 1) < 1e-15
    # ties go to the lowest index, also among groups
    assert router.moe_route_topk(np.zeros((1, 8)), 3, n_group=4, topk_group=2)[0].tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_against_brute_force(score):
    rng = np.random.default_rng(5)
    for _ in range(20):
        x = rng.permutation(np.linspace(-2, 2, 8))[None]
        b = rng.normal(size=8) * 0.1
        c = router.route_choices(x, b, score, 1, 1, 1)[0]
        idx, _ = router.moe_route_topk(x, 3, bias=b, score=score)
        best = max(itertools.combinations(range(8), 3), key=lambda p: sum(c[list(p)]))
        assert sorted(idx[0].tolist()) == list(best)
        assert np.all(np.diff(c[idx[0]]) <= 0)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_against_differences(score, renorm):
    """Central differences with step h = 1e-5 are off by h^2 / 6 times a third
    derivative (about scale) and by 2^-53 / h: together below 1e-9 here."""
    rng = np.random.default_rng(9)
    x = rng.normal(size=(4, 7))
    idx = np.array([[1, 3, 6], [0, -1, 2], [-1, -1, -1], [5, 4, 0]], dtype=np.int32)
    g = rng.normal(size=(4, 3))
    got = router.moe_route_topk_bwd(x, idx, g, score, renorm, 1.5)
    h = 1e-5
    for t in range(4):
        for e in range(7):
            d = np.zeros(7)
            d[e] = h
            up = router.route_weights(x[t] + d, idx[t], score, renorm, 1.5)
            dn = router.route_weights(x[t] - d, idx[t], score, renorm, 1.5)
            assert abs(got[t, e] - (g[t] * (up - dn)).sum() / (2 * h)) < 1e-9
