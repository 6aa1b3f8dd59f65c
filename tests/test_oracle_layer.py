"""Pins of oracle/layer.py: closed forms, central differences, brute force."""

import numpy as np
import pytest

from oracle import layer


def _rng(seed):
    return np.random.default_rng(seed)


def test_norm_closed_forms():
    h = np.array([[3.0, 4.0], [0.0, 0.0], [-7.0, 7.0]])
    y = layer.rms_norm(h, np.array([1.0, 2.0]), 1e-12)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)], [0, 0], [-1, 2]], atol=1e-9)
    # a row scaled by any factor has the same norm
    x = _rng(0).normal(size=(5, 33))
    assert np.allclose(layer.rms_norm(x * 1e3, 1.0, 1e-30), layer.rms_norm(x, 1.0, 1e-30))


def _differences(f, x, dy, step=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        d[i] = ((f(a) - f(b)) * dy).sum() / (2 * step)
    return d


def test_norm_gradients_are_differences():
    r = _rng(1)
    h, w, dy, dh = r.normal(size=(4, 7)), r.normal(size=7), r.normal(size=(4, 7)), r.normal(size=(4, 7))
    dx, dw, size, wsize = layer.rms_norm_bwd(dy, h, w, 1e-2, dh)
    assert np.allclose(dx - dh, _differences(lambda v: layer.rms_norm(v, w, 1e-2), h, dy), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: layer.rms_norm(h, v, 1e-2), w, dy), atol=1e-7)
    assert np.all(size >= np.abs(dx) - 1e-12) and np.all(wsize >= np.abs(dw) - 1e-12)


def test_activation_closed_forms():
    x = np.array([[0.0, 50.0, -800.0, 2.0, 3.0, 4.0], [1.0, -1.0, 800.0, 1.0, 1.0, -1.0]])
    y = layer.swiglu(x, [1.0, 2.0])
    s1 = 1 / (1 + np.exp(-1.0))
    assert np.allclose(y, [[0.0, 150.0, 0.0], [2 * s1, -2 * (1 - s1), -1600.0]], rtol=1e-12, atol=1e-300)


@pytest.mark.parametrize("weighted", [False, True])
def test_activation_gradients_are_differences(weighted):
    r = _rng(2)
    x, dy, w = r.normal(size=(3, 10)) * 2, r.normal(size=(3, 5)), r.uniform(0.1, 2, size=3) if weighted else None
    dx, dw, size, wsize = layer.swiglu_bwd(x, dy, w)
    assert np.allclose(dx, _differences(lambda v: layer.swiglu(v, w), x, dy), atol=1e-7)
    ones = np.ones(3) if w is None else w
    assert np.allclose(dw, _differences(lambda v: layer.swiglu(x, v), ones, dy), atol=1e-7)
    assert np.all(size >= np.abs(dx) - 1e-12) and np.all(wsize >= np.abs(dw) - 1e-12)


def test_ragged_products_by_brute_force():
    r = _rng(3)
    a, b, t = r.normal(size=(9, 4)), r.normal(size=(4, 5, 4)), r.normal(size=(9, 3))
    off = [1, 4, 4, 20, 20]  # row 0 outside, an empty group, an end past the last row, an empty group behind it
    group = [None, 0, 0, 0, 2, 2, 2, 2, 2]
    d, done = layer.ragged_nt(a, b, off)
    e, _ = layer.ragged_nn(a, np.swapaxes(b, 1, 2), off)
    assert done.tolist() == [g is not None for g in group]
    for m, g in enumerate(group):
        for n in range(5):
            want = 0.0 if g is None else sum(a[m, k] * b[g, n, k] for k in range(4))
            assert abs(d[m, n] - want) < 1e-12 and abs(e[m, n] - want) < 1e-12
    c = r.normal(size=(4, 4, 3))
    w = layer.ragged_tn(a, t, off, c)
    for g in range(4):
        for i in range(4):
            for j in range(3):
                assert abs(w[g, i, j] - c[g, i, j] - sum(a[m, i] * t[m, j] for m in range(9) if group[m] == g)) < 1e-12
