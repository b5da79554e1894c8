"""The order in which experts are picked where it is easily lost."""
import numpy as np
import pytest

from _gpu import dev, require_gpu
from test_gpu_moe_ops import check_route, spread_logits

pytestmark = pytest.mark.gpu
LOWEST = np.float32(np.finfo(np.float32).min)


@pytest.mark.parametrize("E,groups", [(16, 4), (60, 5), (256, 8), (64, 32), (1024, 64)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_group_sums_of_masked_biases(E, groups, sigmoid, dtype):
    """Experts masked by a bias of FP32's lowest value: a group with one expert
    left has a larger sum than one with none, whose sum is past the range."""
    require_gpu()
    rng = np.random.default_rng(E)
    t, l = spread_logits(rng, 5, E, dtype)
    size = E // groups
    bias = np.full(E, LOWEST)
    live = groups - 1
    bias[live * size + size // 2] = 0.25
    for topk in (1, 2):
        got, _ = check_route(t, l, topk, sigmoid, bias, groups, 1, True, False, 1.0)
        assert np.all(got[:, 0] == live * size + size // 2)
    bias[(live - 1) * size:(live - 1) * size + 2] = -0.5  # a group with two left comes before that with one
    got, _ = check_route(t, l, 2, sigmoid, bias, groups, 1, True, False, 1.0)
    assert np.all(got // size == live - 1)
    check_route(t, l, 3, sigmoid, bias, groups, 2, True, True, 1.0)


@pytest.mark.parametrize("groups", [1, 4])
def test_values_next_to_the_lowest(groups):
    """Logits and biases between FP32's lowest value and a thousandth above it keep their order."""
    require_gpu()
    E = 32
    l = np.full((3, E), LOWEST)
    l[0, 21] = -3.401e38
    l[1, [5, 30]] = -3.4012e38, -3.4011e38
    l[2, 9] = np.nextafter(LOWEST, np.float32(0))
    for renormalize in (False, True):
        got, w = check_route(dev(l), l, 1, False, None, groups, 1, False, renormalize, 1.0, True)
        assert got[:, 0].tolist() == [21, 30, 9] and np.all(w == 1)
    rng = np.random.default_rng(1)
    t, x = spread_logits(rng, 4, E, "f32")
    bias = np.full(E, np.float32(-3.402e38))
    bias[[11, 23]] = -3.4011e38, -3.401e38
    for sigmoid in (False, True):
        got, _ = check_route(t, x, 2, sigmoid, bias, groups, min(2, groups), False, False, 1.0)
        assert np.all(got == [23, 11])
