"""Expert routing, the weighted combine and their gradients on the GPU against
the 64-bit oracle.  Tolerances follow from FP32 arithmetic: u = 2^-24 per
operation, an exponential's argument x carries |x| u into its relative error,
a sum of N terms at most N u of the sum of their absolute values; BF16
outputs add one rounding of 2^-8 relative."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from oracle import moe_ops
from _gpu import dev, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GUARD = 256


class Out:
    """A device tensor between canaries."""

    def __init__(self, shape, dtype, fill=0):
        n = int(np.prod(shape))
        self.buf = torch.full((n + 2 * GUARD,), 77, dtype=dtype, device="cuda")
        self.view = self.buf[GUARD:GUARD + n].view(shape)
        self.view.fill_(fill)

    def numpy(self):
        torch.cuda.synchronize()
        edge = torch.cat((self.buf[:GUARD], self.buf[self.buf.numel() - GUARD:]))
        assert bool((edge == 77).all()), "written outside the output"
        return self.view.float().cpu().numpy() if self.view.dtype == torch.bfloat16 else self.view.cpu().numpy()


def bf16(a):
    """numpy -> device bfloat16, and the values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def spread_logits(rng, T, E, dtype):
    """Rows of distinct values over [-6, 6], in random order: no two scores
    of a row come within the rounding of either type."""
    grid = np.linspace(-6, 6, E) if E > 1 else np.zeros(1)
    l = np.stack([rng.permutation(grid) for _ in range(T)]).astype(np.float32)
    if dtype == "bf16":
        return bf16(l)
    return dev(l), l


def strided(t, pad):
    """The same values in rows `pad` elements further apart, 9 between them."""
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), 9, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def route_bound(l, ref):
    """|error| of a weight: exponentials' arguments reach twice the largest
    finite |logit| (over 100, they underflow), the sums have E terms."""
    fin = np.abs(np.where(np.isfinite(l), l, 0)).max() if l.size else 0
    return np.abs(ref) * (4 * min(2 * fin, 104.0) + l.shape[1] + 32) * U + 2.0 ** -126


def check_route(t, l, topk, sigmoid=False, bias=None, groups=1, topk_groups=1, top2=False, renormalize=False,
                scale=1.0, all_decided=False):
    T = l.shape[0]
    idx, w = Out((T, topk), torch.int32, 55), Out((T, topk), torch.float32, 55)
    b.fp8_moe_route(t, topk, b.FP8G_SIGMOID if sigmoid else b.FP8G_SOFTMAX, None if bias is None else dev(bias),
                    groups, topk_groups, b.FP8G_GROUP_TOP2 if top2 else b.FP8G_GROUP_MAX, renormalize, scale, idx.view,
                    w.view)
    want_i, want_w, gap = moe_ops.route(l, topk, sigmoid, bias, groups, topk_groups, top2, renormalize, scale)
    # a selection score is at most about 2 (group sums 4) in size; closer than 2^-19, rounding may decide
    decided = np.ones(T, bool) if all_decided else gap > 2.0 ** -19
    assert bias is not None or decided.mean() > 0.8
    got_i, got_w = idx.numpy(), w.numpy()
    assert np.array_equal(got_i[decided], want_i[decided])
    bad = np.abs(got_w - want_w) > route_bound(l, want_w)
    assert not bad[decided].any(), (got_w[bad], want_w[bad])
    return got_i, got_w


ROUTES = [  # T, E, topk, groups, topk_groups, top2
    (1, 1, 1, 1, 1, False), (3, 2, 2, 1, 1, False), (65, 8, 2, 1, 1, False), (7, 16, 16, 1, 1, False),
    (33, 60, 4, 1, 1, False), (130, 64, 6, 1, 1, False), (9, 64, 8, 8, 3, True), (40, 96, 7, 3, 2, False),
    (21, 100, 5, 5, 2, True), (5, 64, 1, 64, 64, True), (12, 130, 10, 13, 4, True), (50, 128, 8, 1, 1, False),
    (17, 256, 8, 8, 4, True), (11, 256, 32, 4, 1, False), (6, 333, 3, 3, 3, True), (4, 1000, 20, 1, 1, False),
    (3, 1024, 8, 32, 9, True), (2, 1024, 32, 1, 1, False), (70, 12, 3, 6, 2, True), (64, 5, 5, 1, 1, False),
]


@pytest.mark.parametrize("T,E,topk,groups,topk_groups,top2", ROUTES)
@pytest.mark.parametrize("dtype,sigmoid,with_bias,renormalize,pad", [
    ("f32", False, False, False, 0), ("bf16", True, True, True, 0), ("f32", True, True, False, 3),
    ("bf16", False, False, True, 8), ("f32", False, True, True, 4), ("bf16", True, False, False, 5)])
def test_route(T, E, topk, groups, topk_groups, top2, dtype, sigmoid, with_bias, renormalize, pad):
    require_gpu()
    rng = np.random.default_rng(T * 1000 + E)
    t, l = spread_logits(rng, T, E, dtype)
    bias = rng.permutation(np.linspace(-0.2, 0.2, E)).astype(np.float32) if with_bias else None
    check_route(strided(t, pad), l, topk, sigmoid, bias, groups, topk_groups, top2, renormalize, 2.5)


@pytest.mark.parametrize("T,E,topk,groups,topk_groups", [
    (3, 1000, 8, 5, 2), (2, 990, 17, 33, 9),  # groups whose padded places outnumber the lanes: 32 experts a lane
    (40000, 8, 2, 1, 1), (9000, 64, 6, 8, 3), (33000, 16, 4, 4, 2), (70001, 4, 3, 1, 1)])  # few lanes a token
def test_route_lane_counts(T, E, topk, groups, topk_groups):
    """Every share of lanes a token can have, against the oracle on a sample of
    rows, and all rows against each other (the rows repeat)."""
    require_gpu()
    rng = np.random.default_rng(T)
    base = 64 if T > 64 else T
    _, l = spread_logits(rng, base, E, "f32")
    reps = -(-T // base)
    full = np.tile(l, (reps, 1))[:T]
    for sigmoid, renormalize in ((False, False), (True, True)):
        idx, w = Out((T, topk), torch.int32, 55), Out((T, topk), torch.float32, 55)
        b.fp8_moe_route(dev(full), topk, b.FP8G_SIGMOID if sigmoid else b.FP8G_SOFTMAX, None, groups, topk_groups,
                        b.FP8G_GROUP_TOP2, renormalize, 1.0, idx.view, w.view)
        gi, gw = idx.numpy(), w.numpy()
        want_i, want_w, gap = moe_ops.route(l, topk, sigmoid, None, groups, topk_groups, True, renormalize)
        ok = gap > 2.0 ** -19
        assert ok.mean() > 0.5 and np.array_equal(gi[:base][ok], want_i[ok])
        assert not (np.abs(gw[:base] - want_w) > route_bound(l, want_w))[ok].any()
        assert np.array_equal(gi, np.tile(gi[:base], (reps, 1))[:T])
        assert np.array_equal(gw, np.tile(gw[:base], (reps, 1))[:T])
        g = rng.normal(size=(base, topk)).astype(np.float32)
        grad = b.fp8_moe_route_backward(dev(full), idx.view, dev(np.tile(g, (reps, 1))[:T]), None,
                                        b.FP8G_SIGMOID if sigmoid else b.FP8G_SOFTMAX, renormalize).cpu().numpy()
        want, mag = moe_ops.route_backward(l, gi[:base], g, sigmoid, renormalize)
        assert np.all(np.abs(grad[:base] - want) <= mag * (8 * 6 + E + 3 * topk + 48) * U + 2.0 ** -126)
        assert np.array_equal(grad, np.tile(grad[:base], (reps, 1))[:T])


def test_combine_backward_of_many_tokens():
    """The form for many tokens, with the weights' gradient and without."""
    require_gpu()
    rng = np.random.default_rng(21)
    T, k, n, rows = 300, 3, 2120, 1000
    dst = pairs(rng, T, k, rows)
    ty, y = bf16(rng.normal(size=(rows, n)))
    tg, go = bf16(rng.normal(size=(T, n)))
    w = rng.normal(size=(T, k)).astype(np.float32)
    for with_gw in (True, False):
        gy, gw = Out((rows, n), torch.bfloat16, 3), Out((T, k), torch.float32, 3)
        b.fp8_moe_combine_backward(tg, ty if with_gw else None, dev(dst), dev(w), gy.view,
                                   gw.view if with_gw else None)
        want_y, want_w, mag = moe_ops.combine_backward(go, y, dst, w, np.full((rows, n), 3.0))
        assert np.all(np.abs(gy.numpy() - want_y) <= np.abs(want_y) * (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * U))
        assert np.all(np.abs(gw.numpy() - want_w) <= (n + 1) * U * mag) if with_gw else np.all(gw.numpy() == 3)


def test_route_ties_go_to_the_lowest_index():
    require_gpu()
    for E, groups, topk in ((8, 1, 3), (256, 8, 8), (100, 5, 5), (1024, 1, 32)):
        for top2 in (False, True):
            l = np.zeros((5, E), np.float32)
            got, w = check_route(dev(l), l, topk, True, None, groups, min(2, groups), top2, True, 1.0, True)
            assert np.array_equal(got, np.tile(np.arange(topk), (5, 1)))
    l = np.repeat(np.float32([[1, 3, 2, 3]]), 64, axis=0)[:, np.arange(64) % 4]
    got, _ = check_route(dev(l), l, 20, False, None, 1, 1, False, False, 1.0, True)
    assert got[0].tolist() == list(range(1, 41, 2))  # sixteen threes from 1 on, and their order
    z = np.float32([[-0.0, 0.0, -0.0, 0.0]])
    got, _ = check_route(dev(z), z, 4, False, None, 1, 1, False, False, 1.0, True)
    assert got.tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masks(dtype, sigmoid, renormalize, groups):
    """Rows masked whole or in part, by -inf, NaN and the type's lowest value;
    infinite logits; biases of -inf and NaN."""
    require_gpu()
    rng = np.random.default_rng(3)
    E, topk = 24, 4
    low = -3.4028235e38 if dtype == "f32" else -3.3895314e38
    _, l = spread_logits(rng, 12, E, dtype)
    l = np.array(l)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 1:] = -np.inf
    l[3, 3:] = np.nan
    l[4] = low
    l[5, ::2] = low
    l[6, 5:] = low
    l[7, :22] = -np.inf
    l[8, 7] = np.inf
    l[9, [3, 20]] = np.inf
    l[10, 6:] = -np.inf  # with groups, all but the first group
    t = dev(l) if dtype == "f32" else bf16(l)[0]
    keep = [r for r in range(12)]
    topk_groups = 1 if groups == 1 else 2
    for bias in (None, np.where(np.arange(E) % 5 == 1, -np.inf, 0).astype(np.float32),
                 np.where(np.arange(E) % 7 == 2, np.nan, 0.25).astype(np.float32)):
        got, w = check_route(t[keep], l[keep], topk, sigmoid, bias, groups, topk_groups, groups > 1, renormalize, 1.5)
        assert np.all(got[0] == -1) and np.all(w[0] == 0) and np.all(got[1] == -1) and np.all(w[1] == 0)
        assert np.all(np.isfinite(w))


def test_route_extreme_bias_stays_in_range():
    require_gpu()
    rng = np.random.default_rng(4)
    t, l = spread_logits(rng, 6, 32, "f32")
    bias = np.where(np.arange(32) == 9, np.inf, np.where(np.arange(32) % 3 == 0, -3.4e38, 3.4e38)).astype(np.float32)
    for top2 in (False, True):
        idx, w = b.fp8_moe_route(t, 4, b.FP8G_SIGMOID, dev(bias), 4, 2,
                                 b.FP8G_GROUP_TOP2 if top2 else b.FP8G_GROUP_MAX)
        idx = idx.cpu().numpy()
        assert np.all((idx >= 0) & (idx < 32)) and all(len(set(r)) == 4 for r in idx.tolist())
        assert np.all(idx[:, 0] == 9)


@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (5, 8, 2), (33, 60, 4), (130, 128, 8), (9, 256, 8), (3, 1000, 32),
                                      (2, 1024, 5), (64, 64, 6), (66, 100, 3)])
@pytest.mark.parametrize("dtype,sigmoid,renormalize,pad", [
    ("f32", False, False, 0), ("f32", False, True, 3), ("f32", True, False, 0), ("f32", True, True, 4),
    ("bf16", False, False, 8), ("bf16", True, True, 0), ("bf16", False, True, 0), ("bf16", True, False, 5)])
def test_route_backward(T, E, topk, dtype, sigmoid, renormalize, pad):
    require_gpu()
    rng = np.random.default_rng(E + topk)
    l = rng.normal(size=(T, E)).astype(np.float32) * 2
    if T > 2:
        l[1, :] = -np.inf
        l[2, rng.integers(0, E, E // 2)] = -np.inf
    t, l = (dev(l), l) if dtype == "f32" else bf16(l)
    idx, _, _ = moe_ops.route(l, topk, sigmoid)
    if T > 4:
        idx[4, 0] = E + 3  # not an expert: counts as none
    g = rng.normal(size=(T, topk)).astype(np.float32)
    want, mag = moe_ops.route_backward(l, idx, g, sigmoid, renormalize, 1.5)
    wide = Out((T, E + pad), t.dtype, 9)
    out = wide.view[:, :E]
    b.fp8_moe_route_backward(strided(t, pad), dev(idx), dev(g), out, b.FP8G_SIGMOID if sigmoid else b.FP8G_SOFTMAX,
                             renormalize, 1.5)
    got = wide.numpy()
    assert np.all(got[:, E:] == 9)
    fin = np.abs(np.where(np.isfinite(l), l, 0)).max()
    bound = mag * (8 * fin + E + 3 * topk + 48) * U + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0) + 2.0 ** -126
    assert np.all(np.abs(got[:, :E] - want) <= bound * (1 + 2.0 ** -8))
    if T > 2:
        assert np.all(got[1, :E] == 0)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_backward_is_the_difference_quotient(sigmoid, renormalize):
    """Against central differences of the 64-bit forward: h = 1e-5 leaves
    under 1e-8, FP32 arithmetic the bound of the test above."""
    require_gpu()
    rng = np.random.default_rng(12)
    T, E, topk, h = 4, 9, 3, 1e-5
    l = rng.normal(size=(T, E)).astype(np.float32)
    g = rng.normal(size=(T, topk)).astype(np.float32)
    idx, _, gap = moe_ops.route(l, topk, sigmoid)
    assert gap.min() > 1e-3
    got = b.fp8_moe_route_backward(dev(l), dev(idx), dev(g), None, b.FP8G_SIGMOID if sigmoid else b.FP8G_SOFTMAX,
                                   renormalize, 2.0).cpu().numpy()
    _, mag = moe_ops.route_backward(l, idx, g, sigmoid, renormalize, 2.0)
    for t, e in np.ndindex(T, E):
        f = []
        for d in (h, -h):
            x = l.astype(np.float64)
            x[t, e] += d
            f.append(np.sum(g * moe_ops.route(x, topk, sigmoid, renormalize=renormalize, scale=2.0)[1]))
        assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) <= 1e-8 + mag[t, e] * (8 * np.abs(l).max() + E + 57) * U


def pairs(rng, T, k, rows):
    """Distinct rows, some pairs dropped (-1, or a row past the end)."""
    d = rng.permutation(max(rows, T * k))[:T * k].reshape(T, k).astype(np.int32)
    d[rng.random((T, k)) < 0.1] = -1
    return d


COMBINES = [(1, 1, 8, 1), (1, 8, 4096, 8), (7, 2, 72, 20), (33, 8, 1000, 300), (130, 4, 2048, 600), (5, 3, 7168, 15),
            (3, 9, 2056, 40), (2, 40, 64, 100), (17, 6, 520, 90)]


@pytest.mark.parametrize("T,k,n,rows", COMBINES)
@pytest.mark.parametrize("mode", ["dst+weights", "weights", "dst", "neither"])
def test_combine(T, k, n, rows, mode):
    require_gpu()
    rng = np.random.default_rng(T + n)
    dst = pairs(rng, T, k, rows) if "dst" in mode else None
    rows = rows if dst is not None else T * k
    ty, y = bf16(rng.normal(size=(rows, n)))
    w = rng.normal(size=(T, k)).astype(np.float32) if "weights" in mode else None
    out = Out((T, n), torch.bfloat16, 5)
    b.fp8_moe_combine(ty, None if dst is None else dev(dst), None if w is None else dev(w), out.view)
    full = np.arange(T * k).reshape(T, k) if dst is None else dst
    want, mag = moe_ops.combine(y, full, np.ones((T, k)) if w is None else w)
    assert np.all(np.abs(out.numpy() - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) + (k + 1) * U * mag * 2)


def test_combine_reads_no_dropped_row():
    """NaN and infinities in rows no pair names, and weights of dropped
    pairs, reach nothing; a token without any pair gets zeros."""
    require_gpu()
    y = torch.full((6, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[2], y[4] = 3.0, float("inf")
    dst = dev(np.int32([[2, -1], [-1, 6], [-7, 2 ** 31 - 1]]))
    w = dev(np.float32([[0.5, np.nan], [np.inf, np.nan], [1, 1]]))
    out = torch.empty(3, 16, dtype=torch.bfloat16, device="cuda")
    b.fp8_moe_combine(y, dst, w, out)
    assert out.float().cpu().numpy().tolist() == [[1.5] * 16, [0.0] * 16, [0.0] * 16]
    gy = torch.full_like(y, 7.0)
    gw = torch.full((3, 2), 9.0, device="cuda")
    b.fp8_moe_combine_backward(torch.ones(3, 16, dtype=torch.bfloat16, device="cuda"), y, dst, w, gy, gw)
    want = np.full((6, 16), 7.0)
    want[2] = 0.5
    assert np.array_equal(gy.float().cpu().numpy(), want)
    assert gw.cpu().numpy().tolist() == [[48.0, 0], [0, 0], [0, 0]]


@pytest.mark.parametrize("T,k,n,rows", COMBINES)
@pytest.mark.parametrize("mode", ["dst+weights", "weights", "dst", "no gradient of the weights"])
def test_combine_backward(T, k, n, rows, mode):
    require_gpu()
    rng = np.random.default_rng(T + n + 1)
    dst = pairs(rng, T, k, rows) if mode != "weights" else None
    rows = rows if dst is not None else T * k
    ty, y = bf16(rng.normal(size=(rows, n)))
    tg, go = bf16(rng.normal(size=(T, n)))
    w = rng.normal(size=(T, k)).astype(np.float32) if mode != "dst" else None
    gy, gw = Out((rows, n), torch.bfloat16, 3), Out((T, k), torch.float32, 3)
    with_gw = mode != "no gradient of the weights"
    b.fp8_moe_combine_backward(tg, ty if with_gw else None, None if dst is None else dev(dst),
                               None if w is None else dev(w), gy.view, gw.view if with_gw else None)
    full = np.arange(T * k).reshape(T, k) if dst is None else dst
    want_y, want_w, mag = moe_ops.combine_backward(go, y, full, np.ones((T, k), np.float32) if w is None else w,
                                                   np.full((rows, n), 3.0))
    # one FP32 product, rounded to BF16
    assert np.all(np.abs(gy.numpy() - want_y) <= np.abs(want_y) * (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * U))
    if with_gw:
        assert np.all(np.abs(gw.numpy() - want_w) <= (n + 1) * U * mag)
    else:
        assert np.all(gw.numpy() == 3)


def test_rows_past_32_bits():
    """A row whose elements start past 2^32 bytes and past 2^31 elements."""
    require_gpu()
    n, rows = 4096, (1 << 31) // 4096 + 3
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    y[rows - 1] = torch.arange(n, device="cuda").remainder(128)
    y[1] = 1.0
    dst = dev(np.int32([[rows - 1, 1]]))
    w = dev(np.float32([[2.0, 1.0]]))
    out = torch.empty(1, n, dtype=torch.bfloat16, device="cuda")
    b.fp8_moe_combine(y, dst, w, out)
    want = 2.0 * (np.arange(n) % 128) + 1
    assert np.array_equal(out.float().cpu().numpy()[0], bf16(want)[1])
    gw = torch.empty(1, 2, device="cuda")
    probe = y[rows - 1].clone()
    b.fp8_moe_combine_backward(torch.ones_like(out), y, dst, w, y, gw)  # in place: each element is read before it is written
    assert np.array_equal(y[rows - 1].float().cpu().numpy(), np.full(n, 2.0))
    assert gw.cpu().numpy().tolist() == [[float(probe.float().sum()), float(n)]]
    del y


def test_another_stream_and_graph_replays():
    """All four calls on a side stream (outputs allocated by the call
    included), and replayed in a graph, with the eager results."""
    require_gpu()
    rng = np.random.default_rng(5)
    T, E, k, n = 40, 64, 4, 256
    t, l = spread_logits(rng, T, E, "f32")
    y = bf16(rng.normal(size=(T * k, n)))[0]
    go = bf16(rng.normal(size=(T, n)))[0]

    def step(stream=None):
        idx, w = b.fp8_moe_route(t, k, renormalize=True, stream=stream)
        out, gy = torch.empty_like(go), torch.empty_like(y)
        gw = torch.empty_like(w)
        b.fp8_moe_combine(y, None, w, out, stream=stream)
        b.fp8_moe_combine_backward(go, y, None, w, gy, gw, stream=stream)
        gl = b.fp8_moe_route_backward(t, idx, gw, renormalize=True, stream=stream)
        return idx, w, out, gy, gw, gl

    ref = [v.clone() for v in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for v in held:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(ref, held))
        step()


def test_binding_refuses_wrong_tensors():
    require_gpu()
    f = lambda *s: torch.zeros(s, device="cuda")
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for bad, err in [
            (lambda: b.fp8_moe_route(f(4, 8).double(), 2), TypeError), (lambda: b.fp8_moe_route(f(4), 2), ValueError),
            (lambda: b.fp8_moe_route(f(8, 4).t(), 2), ValueError),
            (lambda: b.fp8_moe_route(f(1, 8).expand(4, 8), 2), ValueError),
            (lambda: b.fp8_moe_route(torch.zeros(4, 8), 2), TypeError),
            (lambda: b.fp8_moe_route(f(4, 8), 2, bias=f(7)), ValueError),
            (lambda: b.fp8_moe_route(f(4, 8), 2, expert_idx=i(4, 3)), ValueError),
            (lambda: b.fp8_moe_route(f(4, 8), 2, weights=f(3, 2)), ValueError),
            (lambda: b.fp8_moe_route(f(4, 8), 2, weights=h(4, 2)), TypeError),
            (lambda: b.fp8_moe_route_backward(f(4, 8), i(4, 2), f(4, 3)), ValueError),
            (lambda: b.fp8_moe_route_backward(f(4, 8), i(3, 2), f(3, 2)), ValueError),
            (lambda: b.fp8_moe_route_backward(f(4, 8), i(4, 2), f(4, 2), h(4, 8)), TypeError),
            (lambda: b.fp8_moe_combine(h(8, 16), i(4, 2), f(4, 3), h(4, 16)), ValueError),
            (lambda: b.fp8_moe_combine(h(8, 8), i(4, 2), f(4, 2), h(4, 16)), ValueError),
            (lambda: b.fp8_moe_combine(h(7, 16), None, f(4, 2), h(4, 16)), ValueError),
            (lambda: b.fp8_moe_combine(f(8, 16), i(4, 2), f(4, 2), h(4, 16)), TypeError),
            (lambda: b.fp8_moe_combine_backward(h(4, 16), h(7, 16), i(4, 2), f(4, 2), h(8, 16), f(4, 2)), ValueError),
            (lambda: b.fp8_moe_combine_backward(h(4, 16), None, i(4, 2), f(4, 2), h(8, 16), f(4, 2)), ValueError)]:
        with pytest.raises(err):
            bad()
    for bad in (lambda: b.fp8_moe_route(f(4, 8), 9), lambda: b.fp8_moe_route(f(4, 8), 0),
                lambda: b.fp8_moe_route(f(4, 8), 2, score_func=2), lambda: b.fp8_moe_route(f(4, 8), 3, 0, None, 4, 1),
                lambda: b.fp8_moe_route(f(4, 8), 2, 0, None, 3, 1),
                lambda: b.fp8_moe_combine(h(8, 12), i(4, 2), f(4, 2), h(4, 12))):
        with pytest.raises(b.Fp8GemmError):
            bad()


def test_nothing_to_do():
    require_gpu()
    idx, w = b.fp8_moe_route(torch.zeros(0, 8, device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    assert b.fp8_moe_route_backward(torch.zeros(0, 8, device="cuda"), idx, w).shape == (0, 8)
    e = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    b.fp8_moe_combine(e, idx, w, e)
    out = torch.full((3, 16), 4.0, dtype=torch.bfloat16, device="cuda")  # no rows at all: every pair is dropped
    d = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    b.fp8_moe_combine(e, d, None, out)
    assert float(out.float().abs().sum()) == 0
    gw = torch.full((3, 2), 4.0, device="cuda")
    b.fp8_moe_combine_backward(out, e, d, None, e, gw)
    assert float(gw.abs().sum()) == 0
