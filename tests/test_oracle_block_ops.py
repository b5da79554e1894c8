"""The oracle of the feed-forward block against closed forms and differences."""
import numpy as np
import pytest

from oracle import block_ops as o


def test_activations_at_known_points():
    z = np.array([0.0, 1.0, -1.0, 30.0, -np.inf, np.inf])
    assert np.allclose(o.act("gelu", z), [0, 0.8413447460685429, -0.15865525393145707, 30, 0, np.inf])
    assert np.allclose(o.act("silu", z), [0, 0.7310585786300049, -0.2689414213699951, 30, 0, np.inf])
    assert np.allclose(o.act("gelu_tanh", z), [0, 0.8411919906082768, -0.15880800939172324, 30, 0, np.inf])
    assert np.array_equal(o.act("relu", z), [0, 1, 0, 30, 0, np.inf])
    for name in o.ACTS:
        assert np.isnan(o.act(name, np.nan)) and (name == "none" or np.isnan(o.act_grad(name, np.nan)))
        assert o.act_grad(name, np.inf) == 1 and (name == "none" or o.act_grad(name, -np.inf) == 0)


@pytest.mark.parametrize("name", o.ACTS)
def test_activation_gradients_against_differences(name):
    z = np.linspace(-8, 8, 401) + 1e-3
    d = 1e-5
    assert np.allclose(o.act_grad(name, z), (o.act(name, z + d) - o.act(name, z - d)) / (2 * d), atol=1e-8)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post,gate", [(True, "row"), (True, "one"), (False, None), (False, "one"), (True, None)])
def test_norm_gradients_against_differences(layer, post, gate):
    rng = np.random.default_rng(3)
    T, n, eps, scale = 3, 8, 1e-3, 0.7
    p = {"x": rng.normal(size=(T, n)) + 0.3, "residual": rng.normal(size=(T, n)), "pre_weight": rng.normal(size=n)}
    if post:
        p["post_weight"] = rng.normal(size=n)
    if gate:
        p["gate"] = rng.normal(size=(T, n) if gate == "row" else n)
    gh, gy = rng.normal(size=(T, n)), rng.normal(size=(T, n))

    def value(q):
        h, y = o.norm_residual(q["x"], q["residual"], post, q.get("post_weight"), q.get("gate"), scale, q["pre_weight"],
                               layer, eps)
        return (h * gh).sum() + (y * gy).sum(), h

    grads = o.norm_residual_grads(gh, gy, p["x"], value(p)[1], post, p.get("post_weight"), p.get("gate"), scale,
                                  p["pre_weight"], layer, eps)
    for name in p:
        for at in np.ndindex(p[name].shape):
            d = np.zeros_like(p[name])
            d[at] = 1e-6
            slope = (value({**p, name: p[name] + d})[0] - value({**p, name: p[name] - d})[0]) / 2e-6
            assert abs(slope - grads[name][at]) < 1e-6 * (1 + abs(slope)), (name, at)


def test_moe_layer_of_identities():
    """One expert passes x through (G x large, so that its SiLU is G x), one negates it."""
    n = 128
    eye = np.eye(n)
    up = np.stack([np.concatenate([0 * eye, eye]), np.concatenate([0 * eye, eye])])
    up[:, :n, 0] = 64.0  # G x = 64 x_0
    down = np.stack([eye / 64.0, -eye / 64.0])
    x = np.ones((2, n))
    x[1] = 2
    idx, w = np.array([[0, 1], [0, -1]]), np.array([[0.75, 0.25], [0.5, 9.0]])
    out = o.moe_layer(x, idx, w, up, down, "silu")
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 0.5 * 2 * 2)
