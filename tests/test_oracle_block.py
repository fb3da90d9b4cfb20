"""Pins of the oracle's dropout, dense layer and group norm against facts
outside them: the generator's words one by one, the share kept, closed forms,
and central differences for every gradient."""
import math

import numpy as np
import pytest

from oracle import block as ob, lowbit as olb


def test_mask_is_the_generators_halves():
    seed, call, p = (0xABCDEF << 32) | 0x13579, 7, 0.3
    nodes = np.array([0, 3, 2 ** 31 - 1, -1])      # -1 is read as 2^32 - 1
    f = ob.drop_factor(4, 19, p, seed, call, nodes)
    T = 19661                                      # 0.3 * 65536 = 19660.8
    for i, node in enumerate([0, 3, 2 ** 31 - 1, 2 ** 32 - 1]):
        for j in range(19):
            w = int(olb.philox4x32_10(np.array([[j // 8, node, call, 1]], np.uint64),
                                      (seed & 0xFFFFFFFF, seed >> 32))[0, (j % 8) // 2])
            u = (w >> 16) if j % 2 else (w & 0xFFFF)
            assert f[i, j] == (float(np.float32(65536 / (65536 - T))) if u >= T else 0.0)
    # row ids from row0, a prefix of a wider row, and the ends of p
    assert np.array_equal(ob.drop_factor(3, 5, p, seed, call, None, 3), ob.drop_factor(3, 19, p, seed, call, [3, 4, 5])[:, :5])
    assert np.all(ob.drop_factor(2, 9, 0.0, seed) == 1.0) and np.all(ob.drop_factor(2, 9, 1.0, seed) == 0.0)


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_share_kept_and_mean(p):
    f = ob.drop_factor(500, 400, p, 99)
    n = f.size
    assert abs((f > 0).mean() - (1 - p)) < 5 * math.sqrt(p * (1 - p) / n) + 2.0 ** -17
    assert abs(f.mean() - 1.0) < 5 * math.sqrt(p / (1 - p) / n)
    # two calls, two seeds, two rows share no mask
    g = ob.drop_factor(500, 400, p, 99, call=1)
    both = ((f > 0) & (g > 0)).mean()
    assert abs(both - (1 - p) ** 2) < 5 * math.sqrt((1 - p) ** 2 / n)


def test_dropped_values_are_zero():
    f = np.array([[0.0, 2.0]])
    assert np.array_equal(ob.drop(np.array([[np.nan, 3.0]]), f), [[0.0, 6.0]])
    assert np.array_equal(ob.drop(np.array([[np.inf, 3.0]]), f), [[0.0, 6.0]])


@pytest.mark.parametrize("kind", ob.ACTS)
def test_activations(kind):
    z = np.array([-6.0, -1.5, -0.25, 0.25, 1.5, 6.0])
    h = 1e-5
    num = (ob.act(z + h, kind, 0.2) - ob.act(z - h, kind, 0.2)) / (2 * h)
    assert np.allclose(num, ob.act_grad(z, kind, 0.2), atol=1e-8)
    if kind in ("gelu", "silu"):                   # z f(z) with f(z) + f(-z) = 1
        assert np.allclose(ob.act(z, kind) - ob.act(-z, kind), z)
    assert ob.act(np.zeros(1), kind)[0] == 0.0
    assert ob.act_grad(np.zeros(1), kind, 0.2)[0] == {"none": 1.0, "relu": 0.0, "leaky_relu": 0.2, "gelu": 0.5, "silu": 0.5}[kind]


@pytest.mark.parametrize("kind", ob.ACTS)
def test_dense_gradients_by_differences(kind):
    g = np.random.default_rng(5)
    X, W, b = g.standard_normal((6, 4)), g.standard_normal((4, 5)), g.standard_normal(5)
    R, G = g.standard_normal((6, 5)), g.standard_normal((6, 5))
    f = ob.drop_factor(6, 5, 0.4, 3)
    Z, _ = ob.dense_forward(X, W, b, kind, 0.1, f, R)
    assert np.abs(Z).min() > 1e-4                  # no step of the activation within a difference
    _, dW, db, dX = ob.dense_backward(X, W, Z, kind, 0.1, f, G)

    def loss():
        return float((ob.dense_forward(X, W, b, kind, 0.1, f, R)[1] * G).sum())

    for arr, grad in ((X, dX), (W, dW), (b, db)):
        for i in np.ndindex(arr.shape):
            keep, h = arr[i], 1e-6
            arr[i] = keep + h
            up = loss()
            arr[i] = keep - h
            dn = loss()
            arr[i] = keep
            assert abs((up - dn) / (2 * h) - grad[i]) < 1e-6


@pytest.mark.parametrize("groups", [1, 2, 6])
@pytest.mark.parametrize("kind", ["none", "gelu", "leaky_relu"])
def test_norm_gradients_by_differences(groups, kind):
    g = np.random.default_rng(groups)
    X, G = g.standard_normal((11, 6)) * 2 + 3, g.standard_normal((11, 6))
    w, b = g.uniform(0.5, 1.5, 6), g.standard_normal(6)
    seg = [1, 4, 4, 9]                             # rows 0, 9, 10 in no graph, one empty graph
    eps, base = 1e-3, g.standard_normal((11, 6))

    def fwd():
        m, r = ob.norm_stats(X, groups, seg, eps)
        return m, r, ob.norm_forward(X, groups, seg, w, b, kind, 0.1, m, r, base)

    m, r, out = fwd()
    assert np.array_equal(out[[0, 9, 10]], base[[0, 9, 10]])
    G[[0, 9, 10]] = 0.0
    dw, db, dX = ob.norm_backward(X, groups, seg, w, b, kind, 0.1, m, r, G, np.zeros((11, 6)))
    for arr, grad in ((X, dX), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            keep, h = arr[i], 1e-6
            arr[i] = keep + h
            up = float((fwd()[2] * G).sum())
            arr[i] = keep - h
            dn = float((fwd()[2] * G).sum())
            arr[i] = keep
            assert abs((up - dn) / (2 * h) - grad[i]) < 2e-6


def test_norm_of_known_values():
    X = np.array([[1.0, 5.0], [3.0, 9.0], [7.0, 7.0]])
    m, r = ob.norm_stats(X, 2, [0, 2, 3, 3], 0.25)
    assert np.array_equal(m, [[2, 7], [7, 7], [0, 0]])
    assert np.allclose(1 / r ** 2, [[1.25, 4.25], [0.25, 0.25], [0.25, 0.25]])
    m, _ = ob.norm_stats(X, 1, [0, 3], 0.0)
    assert np.isclose(m[0, 0], 32 / 6)
