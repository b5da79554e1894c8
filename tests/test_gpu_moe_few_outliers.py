"""Single large channels in front of the second matrix of the mixture-of-experts
layer for a few tokens: one column of mid in every 128 is 2^13 to 2^27 times its
neighbours (2^34 where all are powers of two), and the second matrix has codes of
0, or its smallest, in that column, so that the output is made of the neighbours.

Tolerances, with u = 2^-24, as in test_gpu_moe_few, but for mid: an FP16 value
with an exponent for each 16 columns is off by 2^-11 of itself (half a step), or,
among FP16's subnormal numbers, by half their step of 2^-24 where the largest of
the 16 lies in 2^14 .. 2^15: by 2^-39 of that.  To be brought to the exponent of
the largest of 128 it is multiplied by two powers of two, each of which may round
once more among the subnormal numbers, and a factor below 2^-38 of the largest
is 0: 2^-37 of the largest of the 128 covers all of it."""
import numpy as np
import pytest
import torch

import oracle
from fp8_block_scaled_04_amd import binding as b
from oracle import block_ops
from _gpu import Guarded, require_gpu
from test_gpu_moe_few import ACT, U, routing, tokens

pytestmark = pytest.mark.gpu


def experts(E, hidden, inter, small, large, at_large, seed):
    """Codes of E experts: G and U with entries of size `small`, and in one row of every 128 of size `large`; D with
    entries of `at_large` in those columns.  ((codes, scales, FP64 matrices) of both matrices, their columns.)"""
    g = torch.Generator().manual_seed(seed)
    table = oracle.e4m3_table()
    code = lambda v: v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    at = torch.randint(0, 128, (E, inter // 128), generator=g) + 128 * torch.arange(inter // 128)
    size = torch.full((E, inter), float(small)).scatter_(1, at, float(large))
    up = code(size.repeat(1, 2)[:, :, None] * torch.randn(E, 2 * inter, hidden, generator=g))
    down = 110 * torch.randn(E, hidden, inter, generator=g)
    down.scatter_(2, at[:, None, :].expand(E, hidden, inter // 128), float(at_large))
    down = code(down)

    def scaled(codes, by):
        E, n, k = codes.shape
        scales = by * torch.exp(0.3 * torch.randn(E, n // 128, k // 128, generator=g))
        exact = np.stack([block_ops.block_matrix(table[codes[e].numpy()], scales[e].numpy()) for e in range(E)])
        return codes.cuda(), scales.cuda(), exact

    return scaled(up, hidden ** -0.5 / small), scaled(down, inter ** -0.5 / 110)


def reference(up, down, x, idx, weights, act):
    """(out, what it may be off by before its rounding, the least ratio of a block's largest to its median), FP64."""
    x = x.double().cpu().numpy()
    I, H = down.shape[2], down.shape[1]
    out, err, ratios = np.zeros((x.shape[0], H)), np.zeros((x.shape[0], H)), []
    for t in range(x.shape[0]):
        for w, e in zip(weights[t].astype(np.float64), idx[t]):
            both = up[e] @ x[t]
            eb = 2 * (H + 64) * U * (np.abs(up[e]) @ np.abs(x[t]))
            g, v = both[:I], both[I:]
            a = block_ops.act(act, g)
            ea = 1.13 * eb[:I] + 2.0 ** -20 * (np.abs(g) + np.abs(a))
            mid = a * v
            em = ea * (np.abs(v) + eb[I:]) + np.abs(a) * eb[I:] + 2 * U * np.abs(mid)
            blocks = np.abs(mid).reshape(-1, 128)
            ratios.append(blocks.max(1) / np.median(blocks, 1))
            near = np.repeat((np.abs(mid) + em).reshape(-1, 128).max(1), 128)
            em = em + 2.0 ** -11 * (np.abs(mid) + em) + 2.0 ** -37 * near
            size = np.abs(down[e]) @ np.abs(mid)
            ey = np.abs(down[e]) @ em + 2 * (I + 64) * U * size
            out[t] += w * (down[e] @ mid)
            err[t] += np.abs(w) * (ey + 64 * U * (size + ey))
    return out, err, np.concatenate(ratios)


# T, topk, E, hidden, inter: a column for each token with 16 and 32 rows a workgroup, tiles of pairs, slices
CASES = [(1, 2, 4, 256, 384), (2, 2, 4, 256, 384), (4, 3, 4, 256, 384), (1, 2, 3, 4224, 128), (3, 1, 3, 4224, 128),
         (12, 2, 4, 256, 384), (64, 2, 4, 256, 384), (9, 1, 3, 4224, 128)]


@pytest.mark.parametrize("small,large,power", [(2, 200, 13), (0.5, 200, 17), (0.1, 150, 20), (0.015, 200, 26)])
@pytest.mark.parametrize("T,topk,E,hidden,inter", CASES)
def test_neighbours_of_a_large_value_keep_theirs(T, topk, E, hidden, inter, small, large, power):
    require_gpu()
    (up, us, up64), (down, ds, down64) = experts(E, hidden, inter, small, large, 0, power)
    idx, w = routing(T, topk, E, T)
    x = tokens(T, hidden, T)
    for act in ("none", "silu"):
        out = Guarded((T, hidden))
        b.fp8_moe_few_tokens(x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), up, us, down, ds, out.view,
                             activation=ACT[act])
        got = oracle.bf16_bits_to_f64(out.result())
        want, err, ratios = reference(up64, down64, x, idx, w, act)
        if act == "none":
            assert np.log2(np.median(ratios)) > power - 1.5  # the inputs are what they are meant to be
        lim = err + 2.0 ** -8 * (np.abs(want) + err)
        assert np.all(np.abs(got - want) <= lim), (act, float((np.abs(got - want) / lim).max()))


@pytest.mark.parametrize("T", [1, 3, 12])
def test_a_large_value_of_little_weight(T):
    """The second matrix's smallest code in the large value's column: both parts of the output count."""
    require_gpu()
    (up, us, up64), (down, ds, down64) = experts(4, 256, 384, 0.5, 200, 2.0 ** -9, 1)
    idx, w = routing(T, 2, 4, T)
    x = tokens(T, 256, T)
    out = Guarded((T, 256))
    b.fp8_moe_few_tokens(x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), up, us, down, ds, out.view)
    got = oracle.bf16_bits_to_f64(out.result())
    want, err, _ = reference(up64, down64, x, idx, w, "silu")
    assert np.all(np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


@pytest.mark.parametrize("T", [1, 4, 16])
def test_factors_down_to_the_last(T):
    """Powers of two throughout, so that nothing rounds before mid is scaled: the largest of 128 is 2^s times its
    neighbours for s up to 34, and the output, from the neighbours alone, is exact."""
    require_gpu()
    hidden, inter = 128, 128
    for s in range(10, 35):
        g = torch.zeros(1, 2 * inter, hidden)  # row r: a power of two in column 0
        a, c = s // 2, s - s // 2
        g[0, :inter, 0], g[0, inter:, 0] = 2.0 ** -9, 2.0 ** -9
        g[0, 37, 0], g[0, inter + 37, 0] = 2.0 ** (a - 9), 2.0 ** (c - 9)
        d = torch.ones(1, hidden, inter)
        d[0, :, 37] = 0
        d[0, 1::2, :100] = 0
        x = torch.zeros(T, hidden, dtype=torch.bfloat16)
        x[:, 0] = 2.0 ** torch.arange(T)
        idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
        code = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        ones = lambda n: torch.full((1, n, 1), 2.0 ** 9, device="cuda")
        out = torch.empty(T, hidden, dtype=torch.bfloat16, device="cuda")
        b.fp8_moe_few_tokens(x.cuda(), idx, None, code(g), ones(2), code(d), torch.ones(1, 1, 1, device="cuda"), out,
                             activation=b.FP8G_ACT_NONE)
        want = torch.empty(T, hidden)
        want[:, 0::2], want[:, 1::2] = 127, 28  # columns but 37; columns from 100 on
        want *= (x[:, :1].float()) ** 2
        assert torch.equal(out.cpu(), want.to(torch.bfloat16)), s
