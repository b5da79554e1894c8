"""Pins of the oracle of expert routing, the weighted combine and the 4-bit
products (oracle/moe_ops.py): hand-computed examples, library routines, and
every gradient against central differences of the forward pass."""
import numpy as np
import pytest

from oracle import moe_ops


def test_route_by_hand():
    """Six experts in three groups: the group with the largest single score
    loses by the sum of two, and the bias picks without weighing."""
    l = np.log(np.array([[4.0, 1.0, 3.0, 2.5, 0.5, 0.25]]))
    p = np.array([4.0, 1.0, 3.0, 2.5, 0.5, 0.25]) / 11.25
    idx, w, _ = moe_ops.route(l, 2)
    assert idx.tolist() == [[0, 2]] and np.allclose(w, p[[0, 2]])
    idx, w, _ = moe_ops.route(l, 2, groups=3, topk_groups=1, top2=True, renormalize=True, scale=2.0)
    assert idx.tolist() == [[2, 3]] and np.allclose(w, [[2 * 3 / 5.5, 2 * 2.5 / 5.5]])
    idx, w, _ = moe_ops.route(l, 2, groups=3, topk_groups=1)
    assert idx.tolist() == [[0, 1]] and np.allclose(w, p[[0, 1]])
    idx, w, _ = moe_ops.route(l, 1, bias=np.array([0, 0, 0, 0, 0, 1.0]))
    assert idx.tolist() == [[5]] and np.allclose(w, p[[5]])


def test_route_without_candidates():
    l = np.array([[-np.inf] * 4, [0.0, -np.inf, np.nan, -np.inf], [1.0, 1.0, 1.0, 1.0]])
    idx, w, _ = moe_ops.route(l, 2, renormalize=True)
    assert idx.tolist() == [[-1, -1], [0, -1], [0, 1]]
    assert w.tolist() == [[0, 0], [1, 0], [0.5, 0.5]]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_is_the_difference_quotient(sigmoid, renormalize):
    rng = np.random.default_rng(7)
    l = rng.normal(size=(3, 10))
    l[1, 4] = -np.inf
    g = rng.normal(size=(3, 4))
    idx, _, gap = moe_ops.route(l, 4, sigmoid, renormalize=renormalize, scale=1.7)
    assert gap.min() > 1e-3  # the steps below change no pick
    got, _ = moe_ops.route_backward(l, idx, g, sigmoid, renormalize, 1.7)
    h = 1e-5
    for t in range(3):
        for e in range(10):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            f = []
            for d in (h, -h):
                x = l.copy()
                x[t, e] += d
                f.append(np.sum(g * moe_ops.route(x, 4, sigmoid, renormalize=renormalize, scale=1.7)[1]))
            # the third derivative times h^2, and the rounding of f over h, are below 1e-9
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) < 1e-8


def test_combine_and_its_gradients():
    rng = np.random.default_rng(8)
    y, w, go = rng.normal(size=(7, 3)), rng.normal(size=(4, 2)), rng.normal(size=(4, 3))
    dst = np.array([[0, 3], [-1, 5], [6, 9], [-1, -1]], np.int32)
    out, _ = moe_ops.combine(y, dst, w)
    assert np.allclose(out[0], w[0, 0] * y[0] + w[0, 1] * y[3])
    assert np.allclose(out[1], w[1, 1] * y[5]) and np.allclose(out[2], w[2, 0] * y[6]) and np.all(out[3] == 0)
    gy, gw, _ = moe_ops.combine_backward(go, y, dst, w, np.zeros_like(y))
    h = 1e-5  # the sums are linear in each argument: differences are exact up to rounding / h
    f = lambda y_, w_: np.sum(go * moe_ops.combine(y_, dst, w_)[0])
    for i in np.ndindex(y.shape):
        d = np.zeros_like(y)
        d[i] = h
        assert abs((f(y + d, w) - f(y - d, w)) / (2 * h) - gy[i]) < 1e-8
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(y, w + d) - f(y, w - d)) / (2 * h) - gw[i]) < 1e-8


def test_w4_by_hand():
    packed = np.array([[0x2F, 0x08], [0x00, 0xF1]], np.uint8)
    assert moe_ops.w4_codes(packed).tolist() == [[15, 2, 8, 0], [0, 0, 1, 15]]
    s = np.array([[0.5, 2.0], [1.0, 1.0]])
    x = np.array([[1.0, 2.0, 4.0, 8.0]])
    # (15-8, 2-8, 8-8, 0-8) * (.5, .5, 2, 2) and (-8, -8, -7, 7)
    assert moe_ops.w4_matvec(x, packed, s)[0].tolist() == [[3.5 - 6 + 0 - 128, -8 - 16 - 28 + 56]]
    z = np.array([[1, 0], [0, 3]], np.uint8)
    assert moe_ops.w4_matvec(x, packed, s, z)[0].tolist() == [[7 + 1 + 64 + 0, 0 + 0 - 8 + 96]]
    # E2M1: -6, 1, -0, 0 and 0, 0, .5, -6
    assert moe_ops.w4_matvec(x, packed, s, e2m1=True)[0].tolist() == [[-3 + 1, 2 - 48]]
    out, _ = moe_ops.w4_matvec_experts(x, np.array([1, 0, -1, 2]), np.stack([packed, packed[::-1]]), np.stack([s, s]))
    assert out[1].tolist() == [-130.5, 4.0] and np.all(out[2:] == 0)
    assert out[0].tolist() == [-4 - 8 - 56 + 112, 7 - 12 + 0 - 64]
