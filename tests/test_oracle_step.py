"""The oracle of the rotation, the routing and the adapters against cases worked
out by hand."""
import math

import numpy as np

import oracle


def test_rotation_by_quarter_turns():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    freq = np.array([math.pi / 2, math.pi])
    y = oracle.rotate_reference(x, [[1]], freq)  # pairs (0, 2) and (1, 3)
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6, 7, 8])
    y = oracle.rotate_reference(x, [[1]], freq, interleaved=True)  # pairs (0, 1) and (2, 3)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6, 7, 8])
    y = oracle.rotate_reference(x, [[0], [1]], freq, axes=[0, 1])
    assert np.allclose(y[0, 0], [1, -2, 3, -4, 5, 6, 7, 8])
    y = oracle.rotate_reference(x, [[0], [1]], freq, axes=[-5, 9])  # limited to the axes there are
    assert np.allclose(y[0, 0], [1, -2, 3, -4, 5, 6, 7, 8])


def test_rotation_keeps_products_of_equal_distances():
    g = np.random.default_rng(0)
    q, k = g.standard_normal((1, 1, 16)), g.standard_normal((1, 1, 16))
    freq = 100.0 ** (-np.arange(8) / 8)
    dot = [float((oracle.rotate_reference(q, [[p]], freq) * oracle.rotate_reference(k, [[p - 3]], freq)).sum())
           for p in (3, 10, 1000)]
    assert np.allclose(dot, dot[0])


def test_routing_of_one_group():
    x = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    e, w = oracle.route_reference(x, 2)
    assert e.tolist() == [[1, 2]] and np.allclose(w, [[4 / 6, 2 / 6]])
    e, w = oracle.route_reference(x, 2, renormalise=False, scale=8)
    assert np.allclose(w, [[4, 2]])
    e, w = oracle.route_reference(x, 4)
    assert e.tolist() == [[1, 2, 0, 3]]  # equal ones by their number
    e, w = oracle.route_reference(x, 1, bias=np.array([0, 0, 0, 9.0]), renormalise=False)
    assert e.tolist() == [[3]] and np.allclose(w, [[1 / 8]])  # the bias chooses, and does not weigh
    e, w = oracle.route_reference(np.zeros((1, 3)), 1, softmax=False, renormalise=False)
    assert e.tolist() == [[0]] and np.allclose(w, [[0.5]])


def test_routing_by_groups():
    x = np.array([[3.0, 0.0, 2.0, 2.0, 2.9, -1.0]])
    assert oracle.route_reference(x, 2, softmax=False, groups=3, keep=1)[0].tolist() == [[0, 1]]
    # two greatest of each: 0.95 + 0.5, 0.88 + 0.88, 0.95 + 0.27
    assert oracle.route_reference(x, 2, softmax=False, groups=3, keep=1, best=2)[0].tolist() == [[2, 3]]
    assert oracle.route_reference(x, 3, softmax=False, groups=3, keep=2, best=2)[0].tolist() == [[0, 2, 3]]


def test_routing_of_what_is_not_there():
    none, nan = -math.inf, math.nan
    x = np.array([[none, 1.0, nan, 1.0], [none, none, nan, none]])
    e, w = oracle.route_reference(x, 3)
    assert e.tolist() == [[1, 3, -1], [-1, -1, -1]] and np.allclose(w, [[0.5, 0.5, 0], [0, 0, 0]])
    e, w = oracle.route_reference(np.zeros((1, 4)), 2, bias=np.array([none, 0, none, nan]), renormalise=False)
    assert e.tolist() == [[1, -1]] and np.allclose(w, [[0.25, 0]])
    e, w = oracle.route_reference(x[:1], 2, groups=2, keep=1)
    assert e.tolist() == [[1, -1]]


def test_adapters():
    y, x = np.ones((3, 2)), np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a, b = np.array([[[1.0, -1.0]]]), np.array([[[2.0], [-3.0]]])
    out, down, up = oracle.adapt_reference(y, x, a, b, [0, -1, 1], [0.5])
    assert np.allclose(out, [[0.0, 2.5], [1, 1], [1, 1]])
    assert np.allclose(down, [[3.0, 4.5], [0, 0], [0, 0]]) and np.allclose(up, [[1.0, 1.5], [0, 0], [0, 0]])
