"""The order in which experts are picked where it is easily lost."""
import numpy as np
import pytest

from fp8_block_scaled_04_amd import binding as b
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


def steps(rng, T, E, lowest):
    """Rows of E consecutive FP32 values from `lowest` on, in random order."""
    first = np.float32(lowest).view(np.int32)
    assert first < 0  # a negative value: its magnitude falls with the bits
    grid = (first - np.arange(E, dtype=np.int32)).view(np.float32)
    return np.stack([rng.permutation(grid) for _ in range(T)])


@pytest.mark.parametrize("lowest", [-0.3, -8.1, -12.5, -30.0, -80.0])
@pytest.mark.parametrize("E,groups", [(64, 1), (256, 1), (96, 4)])
def test_sigmoid_scores_rank_as_their_logits(lowest, E, groups):
    """Without a bias, and with groups by their largest score, adjacent FP32 logits are told apart."""
    require_gpu()
    l = steps(np.random.default_rng(E), 40, E, lowest)
    topk, size = min(32, E // groups), E // groups
    got, _ = b.fp8_moe_route(dev(l), topk, b.FP8G_SIGMOID, None, groups, 1, b.FP8G_GROUP_MAX)
    for t in range(len(l)):
        g = int(np.argmax(l[t].reshape(groups, size).max(1)))
        mine = l[t, g * size:(g + 1) * size]
        assert got[t].cpu().tolist() == (g * size + np.argsort(-mine, kind="stable")[:topk]).tolist()


def test_sigmoid_scores_of_one_and_zero_are_equal():
    """Scores that round to 1 or to 0 in FP32 tie: the lowest index comes first."""
    require_gpu()
    l = np.float32([[18, 40, 3, 1e30, -120, -300, np.inf, LOWEST]])
    got, _ = b.fp8_moe_route(dev(l), 8, b.FP8G_SIGMOID)
    assert got[0].tolist() == [0, 1, 3, 6, 2, 4, 5, 7]


@pytest.mark.parametrize("lowest", [-19.0, -24.5, -31.9, -60.0])
@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8), (100, 5)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_sigmoid_scores_are_as_precise_as_fp32(lowest, E, groups, with_bias):
    """With a bias (of zero, so that the sums are the scores) or with groups by
    the sum of their two largest, ranking takes the scores themselves.  Logits
    below -16 that are adjacent in FP32 are 2^-19 or more apart, and so are
    their scores, relatively.  A score is off by at most 2^-21.4: an ulp each
    (2^-23) of the exponential and the reciprocal, half an ulp each (2^-24) of
    the exponential's correction and of the sum with 1."""
    require_gpu()
    l = steps(np.random.default_rng(E + 1), 40, E, lowest)
    bias = dev(np.zeros(E, np.float32)) if with_bias else None
    score = b.FP8G_GROUP_MAX if with_bias or groups == 1 else b.FP8G_GROUP_TOP2
    size, keep = E // groups, (groups + 1) // 2
    got, _ = b.fp8_moe_route(dev(l), 8, b.FP8G_SIGMOID, bias, groups, keep, score)
    for t in range(len(l)):
        parts = np.sort(1 / (1 + np.exp(-l[t].astype(np.float64))).reshape(groups, size), axis=1)
        sums = parts[:, -1] + (parts[:, -2] if score == b.FP8G_GROUP_TOP2 else 0)
        first = np.argsort(-sums, kind="stable")
        if groups > 1 and sums[first[keep - 1]] - sums[first[keep]] < 2.0 ** -20 * sums[first[0]]:
            continue  # which group stays is left open
        able = np.isin(np.arange(E) // size, first[:keep])
        want = [i for i in np.argsort(-l[t], kind="stable") if able[i]][:8]
        assert got[t].cpu().tolist() == want
