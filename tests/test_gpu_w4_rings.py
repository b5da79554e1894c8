"""4-bit products long enough that every ring in LDS is filled again several
times, for every tile and format, with scales of their own for every row and
group.

Besides the worst-case bound of test_gpu_w4.py, which grows with k, outputs
are held to a statistical one.  With activations of random sign the i-th of G
partial sums of a group is about the root of the sum of its terms' squares in
size, so G roundings (2^-23 each where a rounding may go toward zero) leave an
error of at most 2^-23 sqrt(G A) in the root mean square, A the sum of the
squares of the scaled terms with |code| + |zero|; the k / G additions of group
sums, the zero point's and the split's add 2^-23.5 sqrt((k / G + 16) B), B the
sum of the squares of the scaled terms themselves."""
import numpy as np
import pytest
import torch

import _w4_rules as rules
from fp8_block_scaled_04_amd import binding as b
from oracle import moe_ops
from _gpu import dev, require_gpu
from test_gpu_moe_ops import Out, bf16
from test_gpu_w4 import FMT, check

pytestmark = pytest.mark.gpu
KINDS = [("int4", False), ("int4", True), ("e2m1", False)]


def device_matrix(seed, lead, n, k, group, sdt, with_zeros):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = 0.01 * torch.exp(0.5 * torch.randn(*lead, n, k // group, device="cuda", generator=g))
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, device="cuda", generator=g) if with_zeros else None
    return w, s.to(torch.bfloat16) if sdt == "bf16" else s, z


def check_rows(got, x, w, s, z, e2m1, k):
    """Rows of the matrix (device tensors) against the oracle, by both bounds."""
    w, s, z = w.cpu().numpy(), s.float().cpu().numpy(), None if z is None else z.cpu().numpy()
    want, mag = moe_ops.w4_matvec(x, w, s, z, e2m1)
    check(got, want, mag, k, "f32")
    v, zero, scale = moe_ops.w4_parts(w, s, z, e2m1)
    x2, G = np.asarray(x, np.float64) ** 2, k // s.shape[-1]
    A = x2 @ (((np.abs(v) + zero) * scale) ** 2).T
    B = x2 @ (((v - zero) * scale) ** 2).T
    bound = np.sqrt(np.mean(2.0 ** -46 * G * A + 2.0 ** -47 * (k / G + 16) * B))
    assert np.sqrt(np.mean((got - want) ** 2)) <= bound


def some_rows(rng, n, count=160):
    if n <= count:
        return np.arange(n)
    return np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, count - 2), np.arange(n - 20, n)]))


def refilled(p, times=2):
    return p.blocks >= times * p.depth + 1


# tokens, rows, columns, and what the rules make of them: tile, 16-row operands, split (0: whole rows per wave)
DENSE = [
    (1, 33, 23040, 1, 1, 8), (1, 4500, 12160, 1, 1, 4), (1, 12400, 5760, 1, 1, 2), (1, 24590, 33152, 1, 1, 1),
    (4, 33, 18560, 4, 1, 8), (13, 40, 19200, 4, 1, 8), (3, 4500, 9600, 4, 1, 4), (4, 24600, 8576, 4, 1, 1),
    (8, 2060, 14720, 8, 1, 8), (5, 2111, 15360, 8, 1, 8),
    (16, 2060, 7296, 16, 1, 8), (9, 2900, 8192, 16, 1, 8),
    (33, 1400, 7424, 16, 2, 8), (16, 9000, 3968, 16, 2, 4), (64, 6200, 2176, 16, 2, 2), (64, 12300, 2304, 16, 2, 1),
    (1, 24600, 2688, 1, 1, 0), (4, 24600, 2176, 4, 1, 0), (16, 49200, 1152, 16, 2, 0)]


@pytest.mark.parametrize("m,n,k,tile,operands,split", DENSE)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fmt,with_zeros", KINDS)
def test_long_products(m, n, k, tile, operands, split, group, fmt, with_zeros):
    require_gpu()
    p = rules.plan(m, n, k, group, with_zeros)
    assert (p.tokens, p.rows, 0 if p.streamed else p.split) == (tile, operands, split) and refilled(p), p
    rng = np.random.default_rng(n + k)
    w, s, z = device_matrix(n + k, (), n, k, group, "bf16" if group == 64 else "f32", with_zeros)
    tx, x = bf16(rng.normal(size=(m, k)))
    out = Out((m, n), torch.float32, 5)
    b.fp8_w4_matvec(tx, w, s, out.view, FMT[fmt], z)
    rows = some_rows(rng, n)
    check_rows(out.numpy()[:, rows], x, w[rows], s[rows], None if z is None else z[rows], fmt == "e2m1", k)


# pairs a token, experts, ... as above
ROUTED = [
    (1, 2, 16, 33, 23040, 1, 1, 8), (2, 4, 64, 1600, 5760, 1, 1, 2), (1, 8, 64, 3100, 2688, 1, 1, 0),
    (4, 2, 8, 33, 18560, 4, 1, 8), (8, 4, 32, 400, 4864, 4, 1, 2), (8, 8, 64, 500, 2176, 4, 1, 0),
    (20, 4, 5, 200, 7296, 16, 1, 8), (40, 2, 4, 800, 8192, 16, 1, 8),
    (20, 8, 9, 500, 7424, 16, 2, 8), (40, 8, 24, 700, 4096, 16, 2, 4), (50, 2, 24, 1500, 2304, 16, 2, 2),
    (50, 4, 24, 2050, 2304, 16, 2, 1), (50, 4, 24, 2050, 2048, 16, 2, 0)]


@pytest.mark.parametrize("T,topk,E,n,k,tile,operands,split", ROUTED)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fmt,with_zeros", KINDS)
def test_long_products_of_experts(T, topk, E, n, k, tile, operands, split, group, fmt, with_zeros):
    require_gpu()
    p = rules.plan(T * topk, n, k, group, with_zeros, E)
    assert (p.tokens, p.rows, 0 if p.streamed else p.split) == (tile, operands, split) and refilled(p), p
    rng = np.random.default_rng(n + k)
    e = rng.integers(-1 if T > 1 else 0, E, (T, topk)).astype(np.int32)
    w, s, z = device_matrix(n + k, (E,), n, k, group, "bf16" if group == 64 else "f32", with_zeros)
    tx, x = bf16(rng.normal(size=(T, k)))
    out = Out((T * topk, n), torch.float32, 5)
    b.fp8_w4_matvec_experts(tx, dev(e), w, s, out.view, FMT[fmt], z)
    got, rows, e = out.numpy(), some_rows(rng, n, 60), e.reshape(-1)
    assert np.all(got[e < 0] == 0)
    for g in sorted(set(e[e >= 0].tolist())):
        pairs = np.nonzero(e == g)[0]
        check_rows(got[np.ix_(pairs, rows)], x[pairs // topk], w[g, rows], s[g, rows], None if z is None else z[g, rows],
                   fmt == "e2m1", k)


@pytest.mark.parametrize("m,n,k,E", [(1, 524400, 1280, None), (4, 524300, 1376, None), (16, 1048600, 640, None),
                                     (140, 16400, 672, 64)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("fmt,with_zeros", KINDS)
def test_streams_of_several_row_sets(m, n, k, E, group, fmt, with_zeros):
    """A wave's ring runs on from one set of rows into the next."""
    require_gpu()
    k = k // group * group
    p = rules.plan(m, n, k, group, with_zeros, E)
    assert p.streamed and p.blocks >= 2 * p.per_set and p.per_set > p.depth and refilled(p), p
    rng = np.random.default_rng(n)
    lead = () if E is None else (E,)
    w, s, z = device_matrix(n, lead, n, k, group, "f32", with_zeros)
    tx, x = bf16(rng.normal(size=(m, k)))
    out = Out((m, n), torch.float32, 5)
    rows = some_rows(rng, n, 400)
    if E is None:
        b.fp8_w4_matvec(tx, w, s, out.view, FMT[fmt], z)
        check_rows(out.numpy()[:, rows], x, w[rows], s[rows], None if z is None else z[rows], fmt == "e2m1", k)
        return
    e = rng.integers(0, E, m).astype(np.int32)
    b.fp8_w4_matvec_experts(tx, dev(e), w, s, out.view, FMT[fmt], z)
    got = out.numpy()
    for g in sorted(set(e.tolist()))[::7]:
        pairs = np.nonzero(e == g)[0]
        check_rows(got[np.ix_(pairs, rows)], x[pairs], w[g, rows], s[g, rows], None if z is None else z[g, rows],
                   fmt == "e2m1", k)


@pytest.mark.parametrize("E,n,k,group,topk", [(140, 16384, 4096, 64, 2), (70, 8192, 16384, 128, 1)])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_scales_of_experts_past_32_bits(E, n, k, group, topk, fmt):
    """Experts whose codes start past 2^32 bytes, each with its own scales."""
    require_gpu()
    rng = np.random.default_rng(k)
    w = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, n, k // group, device="cuda")
    for i, g in enumerate((0, E - 1)):
        w[g], s[g], _ = device_matrix(i, (), n, k, group, "f32", False)
    tx, x = bf16(rng.normal(size=(2, k)))
    e = np.int32([[E - 1, 0], [0, E - 1]])[:, :topk]
    out = torch.empty(2 * topk, n, device="cuda")
    b.fp8_w4_matvec_experts(tx, dev(e), w, s, out, FMT[fmt])
    rows = some_rows(rng, n, 300)
    for p, g in enumerate(e.reshape(-1).tolist()):
        check_rows(out[p, rows].cpu().numpy()[None], x[p // topk:p // topk + 1], w[g, rows], s[g, rows], None,
                   fmt == "e2m1", k)
