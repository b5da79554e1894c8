"""The mixture-of-experts layer for a few tokens on the GPU against the 64-bit
oracle.  Tolerances, with u = 2^-24: a sum of N products formed in FP32 is off by
2 N u of the sum of their absolute values (2: the matrix cores may truncate);
an activation by 2^-20 of |z| + |act(z)| on top, and no slope exceeds 1.13; mid is
rounded to FP16, 2^-11 of its value or 2^-25 of the largest of 128 neighbours
(what lies under 2^-14 of that may be dropped: 2^-14 at most of what has 2^-11 of
the largest's own); the output to BF16, 2^-8."""
import numpy as np
import pytest
import torch

import oracle
from fp8_block_scaled_04_amd import binding as b
from oracle import block_ops
from _gpu import Guarded, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACT = {"none": b.FP8G_ACT_NONE, "relu": b.FP8G_ACT_RELU, "gelu": b.FP8G_ACT_GELU, "gelu_tanh": b.FP8G_ACT_GELU_TANH,
       "silu": b.FP8G_ACT_SILU}
_layers = {}


class Layer:
    """Codes and scales of E experts, and the FP64 matrices they stand for."""

    def __init__(self, E, hidden, inter, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.E, self.hidden, self.inter = E, hidden, inter
        table = oracle.e4m3_table()

        def make(n, k):
            codes = (110 * torch.randn(E, n, k, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            scales = k ** -0.5 / 110 * torch.exp(0.3 * torch.randn(E, n // 128, k // 128, generator=g))
            exact = np.stack([block_ops.block_matrix(table[codes[e].numpy()], scales[e].numpy()) for e in range(E)])
            return codes.cuda(), scales.cuda(), exact

        self.up, self.up_scales, self.up64 = make(2 * inter, hidden)
        self.down, self.down_scales, self.down64 = make(hidden, inter)


def layer(E, hidden, inter):
    key = (E, hidden, inter)
    if key not in _layers:
        _layers[key] = Layer(*key)
    return _layers[key]


def reference(m, x, idx, weights, act):
    """(out, what it may be off by before its rounding), FP64."""
    x = x.double().cpu().numpy()
    I, H = m.inter, m.hidden
    out, err = np.zeros((x.shape[0], H)), np.zeros((x.shape[0], H))
    for t in range(x.shape[0]):
        for j, e in enumerate(idx[t]):
            if not 0 <= e < m.E:
                continue
            w = 1.0 if weights is None else float(weights[t, j])
            both = m.up64[e] @ x[t]
            eb = 2 * (H + 64) * U * (np.abs(m.up64[e]) @ np.abs(x[t]))
            g, v = both[:I], both[I:]
            a = block_ops.act(act, g)
            ea = 1.13 * eb[:I] + 2.0 ** -20 * (np.abs(g) + np.abs(a))
            mid = a * v
            em = ea * (np.abs(v) + eb[I:]) + np.abs(a) * eb[I:] + 2 * U * np.abs(mid)
            near = np.repeat((np.abs(mid) + em).reshape(-1, 128).max(1), 128)
            em = em + 2.0 ** -11 * (np.abs(mid) + em) + 2.0 ** -25 * near
            y = m.down64[e] @ mid
            size = np.abs(m.down64[e]) @ np.abs(mid)
            ey = np.abs(m.down64[e]) @ em + 2 * (I + 64) * U * size
            out[t] += w * y
            err[t] += np.abs(w) * (ey + 64 * U * (size + ey))
    return out, err


def check(m, x, idx, weights, act="silu", workspace=None):
    T = x.shape[0]
    out = Guarded((T, m.hidden))
    i = torch.from_numpy(np.ascontiguousarray(idx, dtype=np.int32)).cuda()
    w = None if weights is None else torch.from_numpy(np.ascontiguousarray(weights, dtype=np.float32)).cuda()
    b.fp8_moe_few_tokens(x, i, w, m.up, m.up_scales, m.down, m.down_scales, out.view, activation=ACT[act],
                         workspace=workspace)
    bits = out.result()
    got = oracle.bf16_bits_to_f64(bits)
    want, err = reference(m, x, np.asarray(idx), weights, act)
    bad = np.abs(got - want) > err + 2.0 ** -8 * (np.abs(want) + err)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    return bits


def tokens(T, hidden, seed, pad=0):
    x = torch.randn(T, hidden + pad, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    return x[:, :hidden]


def routing(T, topk, E, seed):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:topk] for _ in range(T)]).astype(np.int32)
    return idx, rng.uniform(0.05, 1, (T, topk)).astype(np.float32)


# T, topk, E, hidden, inter: a column for each token and tiles of pairs; the second kernel by 16 and 32 rows, whole and in
# slices; fewer 128-column blocks than waves; several launches
CASES = [(1, 1, 1, 128, 128), (1, 8, 8, 512, 384), (2, 3, 8, 256, 128), (3, 2, 8, 512, 384), (4, 8, 8, 512, 384),
         (1, 2, 3, 4224, 128), (4, 1, 3, 4224, 128), (5, 2, 8, 512, 384), (6, 1, 3, 4224, 128), (8, 8, 8, 512, 384),
         (16, 2, 40, 256, 640), (17, 4, 40, 256, 640), (30, 6, 8, 512, 384), (64, 8, 8, 512, 384), (64, 1, 1, 128, 128),
         (65, 3, 8, 256, 128), (130, 2, 8, 256, 128), (7, 3, 4, 1024, 1024), (40, 2, 4, 1024, 1024), (2, 3, 4, 1024, 1024)]


@pytest.mark.parametrize("T,topk,E,hidden,inter", CASES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_layer(T, topk, E, hidden, inter, act):
    require_gpu()
    idx, w = routing(T, topk, E, T)
    check(layer(E, hidden, inter), tokens(T, hidden, T, pad=0 if act == "silu" else 8), idx, w, act)


@pytest.mark.parametrize("act", block_ops.ACTS)
@pytest.mark.parametrize("T", [2, 9])
def test_activations(act, T):
    require_gpu()
    idx, w = routing(T, 2, 8, 5)
    check(layer(8, 256, 128), tokens(T, 256, 5), idx, w, act)


@pytest.mark.parametrize("T", [1, 4, 5, 20, 64])
def test_dropped_repeated_and_foreign_picks(T):
    """-1 and indices past the experts add nothing; a token without any expert gets zeros; an expert named twice or more
    counts with the sum of its weights; no weights are ones."""
    require_gpu()
    m = layer(8, 256, 128)
    rng = np.random.default_rng(T)
    idx = rng.integers(-2, 10, (T, 6)).astype(np.int32)
    idx[0] = [3, 3, -1, 3, 3, 8]
    idx[T // 2] = -1
    if T == 1:
        idx[0] = [5, 2, 5, 2, 5, 1 << 30]
    w = rng.uniform(-1, 1, idx.shape).astype(np.float32)
    bits = check(m, tokens(T, 256, T), idx, w)
    if T > 1:
        assert not bits[T // 2].any()
    check(m, tokens(T, 256, T), idx, None)
    none = np.full((T, 6), -1, np.int32)
    assert not check(m, tokens(T, 256, T), none, w).any()


@pytest.mark.parametrize("T", [16, 17, 50, 64])
def test_one_expert_takes_all(T):
    """Tiles of 16 pairs, full ones and a rest, beside experts with a pair each."""
    require_gpu()
    m = layer(40, 256, 640)
    idx = np.stack([np.full(T, 7), np.arange(T) % 33 + 7], 1).astype(np.int32)  # token 0, 33: 7 twice
    check(m, tokens(T, 256, 1), idx, routing(T, 2, 40, 2)[1])


def test_many_picks_a_token():
    """32 picks: 16 tokens a launch."""
    require_gpu()
    for T in (1, 4, 16, 37):
        idx, w = routing(T, 32, 40, T)
        check(layer(40, 256, 640), tokens(T, 256, T), idx, w / 8)


@pytest.mark.parametrize("T", [3, 24])
def test_equal_calls_equal_bits_whatever_the_workspace_held(T):
    require_gpu()
    m = layer(4, 1024, 1024)
    idx, w = routing(T, 3, 4, T)
    x = tokens(T, 1024, T)
    need = b.fp8_moe_few_tokens_workspace_bytes(T, 3, 1024, 1024)
    first = check(m, x, idx, w)
    for fill in (0, 255, 0x5A):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert np.array_equal(check(m, x, idx, w, workspace=ws), first)
    # a workspace that other shapes, and the split-K GEMM, have used
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    small = layer(8, 256, 128)
    i2, w2 = routing(40, 4, 8, 1)
    q = torch.randint(0, 100, (64, 2048), dtype=torch.uint8, device="cuda")
    qw = torch.randint(0, 100, (256, 2048), dtype=torch.uint8, device="cuda")
    out = torch.empty(64, 256, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        check(small, tokens(40, 256, 3), i2, w2, workspace=ws)
        b.fp8_gemm_nt(q, torch.ones(16, 64, device="cuda"), qw, torch.ones(2, 16, device="cuda"), out, workspace=ws)
        assert np.array_equal(check(m, x, idx, w, workspace=ws), first)


def test_small_and_large_values():
    """Activations far from one: mid's exponents follow, also where a row's values differ by 2^40."""
    require_gpu()
    m = layer(8, 256, 128)
    for T in (2, 12):
        idx, w = routing(T, 2, 8, 9)
        base = tokens(T, 256, 9)
        for size in (2.0 ** -20, 2.0 ** 15):
            check(m, (base.float() * size).bfloat16(), idx, w, "relu")
        mixed = base.clone()
        mixed[:, ::2] *= 2.0 ** -40
        check(m, mixed, idx, w, "none")
        # the products of a block pass FP32's range before its scale, the values do not
        big = Layer(8, 256, 128, seed=3)
        big.up_scales *= 2.0 ** -100
        big.up64 = big.up64 * 2.0 ** -100
        check(big, (base.float() * 2.0 ** 118).bfloat16(), idx, w, "none")


def test_nan_and_infinity_stay_with_their_token():
    require_gpu()
    m = layer(8, 512, 384)
    for T in (3, 4, 20):
        idx, w = routing(T, 4, 8, T)
        x = tokens(T, 512, T).contiguous()
        clean = check(m, x, idx, w)
        dirty = x.clone()
        dirty[1, 7], dirty[2, 3] = torch.nan, torch.inf
        out = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
        b.fp8_moe_few_tokens(dirty, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), m.up, m.up_scales, m.down,
                             m.down_scales, out)
        bits = out.view(torch.int16).cpu().numpy().view(np.uint16)
        rest = [t for t in range(T) if t not in (1, 2)]
        assert np.array_equal(bits[rest], clean[rest])
        assert bool(torch.isnan(out[1]).all()) and not bool(torch.isfinite(out[2]).any())


def test_other_streams_and_a_graph():
    require_gpu()
    m = layer(8, 512, 384)
    for T in (1, 30):
        idx, w = routing(T, 4, 8, T)
        i, wt, x = torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), tokens(T, 512, T).contiguous()
        want = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
        run = lambda out, **kw: b.fp8_moe_few_tokens(x, i, wt, m.up, m.up_scales, m.down, m.down_scales, out, **kw)
        run(want)
        torch.cuda.synchronize()
        outs = [torch.zeros_like(want) for _ in range(3)]
        streams = [torch.cuda.Stream() for _ in outs]
        for o, s in zip(outs, streams):  # two calls at once, a workspace each
            run(o, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        ws = torch.empty(b.fp8_moe_few_tokens_workspace_bytes(T, 4, 512, 384), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)
        with torch.cuda.stream(streams[0]):
            run(out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(out, workspace=ws)
        for k in range(4):  # each with other inputs in the same places
            x.copy_(tokens(T, 512, 100 + k))
            i.copy_(torch.from_numpy(routing(T, 4, 8, 100 + k)[0]))
            run(want)
            out.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_binding_refuses_what_does_not_fit():
    require_gpu()
    m = layer(8, 256, 128)
    idx, w = (torch.from_numpy(t).cuda() for t in routing(4, 2, 8, 1))
    good = dict(x=tokens(4, 256, 1), expert_idx=idx, weights=w, up=m.up, up_scales=m.up_scales, down=m.down,
                down_scales=m.down_scales, out=torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"))
    f = lambda **o: b.fp8_moe_few_tokens(**{**good, **o})
    f()
    f(up=m.up.view(torch.float8_e4m3fn), down=m.down.view(torch.float8_e4m3fn))
    for bad in (dict(expert_idx=idx[:3]), dict(weights=w[:, :1]), dict(up=m.up[:7]), dict(up_scales=m.up_scales[:, :1]),
                dict(down=m.down[:, :128]), dict(down_scales=m.down_scales[:7]), dict(out=good["out"][:3]),
                dict(x=tokens(4, 128, 1)), dict(x=good["x"].t()), dict(expert_idx=idx.view(-1))):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(x=good["x"].float()), dict(expert_idx=idx.long()), dict(weights=w.bfloat16()), dict(out=good["out"].float()),
                dict(up=m.up.float()), dict(up_scales=m.up_scales.double()), dict(out=good["out"].cpu())):
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(b.Fp8GemmError):
        f(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(b.Fp8GemmError):
        f(activation=9)
