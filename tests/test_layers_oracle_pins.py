"""Pins of the fp64 layer oracle: closed forms, hand-worked values, and every gradient against
central differences of its own forward function."""
import math

import numpy as np
import pytest

from oracle import layers_oracle as lo


def central(f, x, h=1e-5):
    """Gradient of the scalar f at x by central differences (error about h^2)."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_activation_values():
    assert lo.act(-2.0, "relu") == 0 and lo.act(3.0, "relu") == 3
    assert lo.act(-2.0, "relu2") == 0 and lo.act(3.0, "relu2") == 9
    phi1 = 0.5 * (1 + math.erf(1 / math.sqrt(2)))
    assert abs(lo.act(1.0, "gelu") - phi1) < 1e-15
    assert abs(lo.act(-1.0, "gelu") + (1 - phi1)) < 1e-15
    u = math.sqrt(2 / math.pi) * 1.044715
    assert abs(lo.act(1.0, "gelu_tanh") - 0.5 * (1 + math.tanh(u))) < 1e-15
    assert abs(lo.act(1.0, "silu") - 1 / (1 + math.exp(-1))) < 1e-15


@pytest.mark.parametrize("name", lo.ACTS)
def test_activation_slopes_are_differences(name):
    z = np.array([-6.0, -2.5, -1.0, -0.3, 0.2, 0.9, 1.7, 4.0, 8.0])
    h = 1e-5
    d = (lo.act(z + h, name) - lo.act(z - h, name)) / (2 * h)
    assert np.allclose(lo.act_slope(z, name), d, atol=1e-9)


def test_layer_norm_by_hand():
    y, mean, rstd = lo.layer_norm([[1.0, 2.0, 3.0, 6.0]], [2.0, 1, 1, 1], [0, 0, 0, 10.0], eps=0.0)
    r = 1 / math.sqrt(3.5)  # variance (4 + 1 + 0 + 9) / 4
    assert mean[0] == 3 and abs(rstd[0] - r) < 1e-15
    assert np.allclose(y, [[-4 * r, -r, 0, 3 * r + 10]], atol=1e-15)


def test_layer_norm_gradients_are_differences():
    rng = np.random.default_rng(0)
    x, dy, gain, bias = rng.normal(size=(3, 5)), rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=5)
    skip = rng.normal(size=(3, 5))

    def loss(x_, g_, b_):
        return (lo.layer_norm(x_, g_, b_)[0] * dy).sum() + (skip * x_).sum()

    _, mean, rstd = lo.layer_norm(x, gain, bias)
    dx, dg, db = lo.layer_norm_backward(dy, x, mean, rstd, gain, skip)
    assert np.allclose(dx, central(lambda v: loss(v, gain, bias), x), atol=1e-8)
    assert np.allclose(dg, central(lambda v: loss(x, v, bias), gain), atol=1e-8)
    assert np.allclose(db, central(lambda v: loss(x, gain, v), bias), atol=1e-8)


@pytest.mark.parametrize("name", lo.ACTS)
def test_linear_gradients_are_differences(name):
    """Two layers: the second's dx, with the first's activation folded in, is the first's dz."""
    rng = np.random.default_rng(1)
    x, w1, b1 = rng.normal(size=(3, 4)), rng.normal(size=(5, 4)), rng.normal(size=5)
    w2, b2, r, dy = rng.normal(size=(2, 5)), rng.normal(size=2), rng.normal(size=(3, 2)), rng.normal(size=(3, 2))

    def loss(x_, w1_, b1_, w2_, b2_):
        h_, _ = lo.linear(x_, w1_, b1_, name)
        return (lo.linear(h_, w2_, b2_, "none", r)[0] * dy).sum()

    h, z = lo.linear(x, w1, b1, name)
    dz, dw2, db2 = lo.linear_backward(dy, h, w2, name, z)
    dx, dw1, db1 = lo.linear_backward(dz, x, w1)
    for got, k in ((dx, 0), (dw1, 1), (db1, 2), (dw2, 3), (db2, 4)):
        args = [x, w1, b1, w2, b2]

        def f(v):
            a = list(args)
            a[k] = v
            return loss(*a)

        assert np.allclose(got, central(f, args[k]), atol=1e-7)


def test_linear_by_hand():
    y, z = lo.linear([[1.0, 2.0]], [[3.0, 4.0], [-1.0, 0.0]], [0.5, 0.25], "relu", [[10.0, 20.0]])
    assert np.array_equal(z, [[11.5, -0.75]]) and np.array_equal(y, [[21.5, 20.0]])
    dx, dw, db = lo.linear_backward([[2.0, 1.0]], [[1.0, 2.0]], [[3.0, 4.0], [-1.0, 0.0]], "relu", [[1.0, -1.0]],
                                    [[0.0, 7.0]])
    assert np.array_equal(dx, [[5.0, 7.0]]) and np.array_equal(dw, [[2.0, 4.0], [1.0, 2.0]])
    assert np.array_equal(db, [2.0, 1.0])
