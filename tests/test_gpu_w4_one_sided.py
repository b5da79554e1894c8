"""INT4 products of activations that share a sign.  A group's result is the
difference scale (sum code x - zero sum x), two sums that are then several
times its size, so its rounding goes by terms of |code| + zero, as the header
says.

Bound on the root mean square: the partial sums of a group of G are at most
S = sum (|code| + zero) |x| scale, G roundings of 2^-23 at most, independent of
each other, leave 2^-23 sqrt(G) S, and groups add in squares; the k / G
additions of group sums, the zero points' and the split's add
2^-23.5 sqrt((k / G + 16) B), B the sum of the squares of the scaled terms."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from oracle import moe_ops
from _gpu import dev, require_gpu
from test_gpu_moe_ops import Out, bf16

pytestmark = pytest.mark.gpu


def activations(rng, kind, m, k):
    n = rng.normal(size=(m, k))
    return {"positive": np.abs(n), "negative": -np.abs(n), "offset": 5 + 0.1 * n, "one value": np.full((m, k), 3.1)}[kind]


@pytest.mark.parametrize("m,n,k", [(1, 100, 7168), (4, 64, 2048), (8, 2060, 1152), (16, 2060, 1152), (33, 1400, 1152),
                                   (16, 49200, 256)])
@pytest.mark.parametrize("kind", ["positive", "negative", "offset", "one value"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("with_zeros", [False, True])
@pytest.mark.parametrize("codes", ["rounded normals", "nearly all zero"])
def test_one_sided_activations(m, n, k, kind, group, with_zeros, codes):
    require_gpu()
    rng = np.random.default_rng(m + k)
    zeros = rng.integers(5, 12, (n, k // group), dtype=np.uint8) if with_zeros else None
    middle = np.full((n, k), 8) if zeros is None else np.repeat(zeros, group, axis=1)
    if codes == "nearly all zero":  # codes at the zero point but one in 50
        c = np.where(rng.random((n, k)) < 0.02, rng.integers(0, 16, (n, k)), middle)
    else:
        c = np.clip(np.rint(middle + 2.6 * rng.normal(size=(n, k))), 0, 15)
    c = c.astype(np.uint8)
    packed = c[:, 0::2] | (c[:, 1::2] << 4)
    s = (0.01 * np.exp(0.5 * rng.normal(size=(n, k // group)))).astype(np.float32)
    tx, x = bf16(activations(rng, kind, m, k))
    out = Out((m, n), torch.float32, 5)
    b.fp8_w4_matvec(tx, dev(packed), dev(s), out.view, zeros=None if zeros is None else dev(zeros))
    rows = np.unique(rng.integers(0, n, 200))
    want, _ = moe_ops.w4_matvec(x, packed[rows], s[rows], None if zeros is None else zeros[rows])
    v, zero, scale = moe_ops.w4_parts(packed[rows], s[rows], None if zeros is None else zeros[rows], False)
    S = np.einsum("mgc,ngc->mng", np.abs(x.astype(np.float64)).reshape(m, -1, group),
                  ((v + zero) * scale).reshape(len(rows), -1, group), optimize=True)
    B = (x.astype(np.float64) ** 2) @ (((v - zero) * scale) ** 2).T
    bound = np.sqrt(np.mean(2.0 ** -46 * group * (S ** 2).sum(-1) + 2.0 ** -47 * (k / group + 16) * B))
    assert np.sqrt(np.mean((out.numpy()[:, rows] - want) ** 2)) <= bound
