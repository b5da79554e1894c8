"""4-bit products: a token's bits do not depend on the other tokens' values,
on its own place among them, or, by experts, on where its pair stands in its
expert's tiles.  (On the number of tokens they do, through the split of k.)"""
import numpy as np
import pytest
import torch

import _w4_rules as rules
from fp8_block_scaled_04_amd import binding as b
from _gpu import dev, require_gpu
from test_gpu_moe_ops import bf16
from test_gpu_w4 import FMT
from test_gpu_w4_rings import device_matrix

pytestmark = pytest.mark.gpu
KINDS = [("int4", False, torch.float32), ("int4", True, torch.bfloat16), ("e2m1", False, torch.float32)]


@pytest.mark.parametrize("m,n,k,tile,streamed", [
    (3, 100, 2304, 4, False), (11, 90, 1152, 4, False), (4, 25000, 256, 4, True), (8, 2060, 640, 8, False),
    (16, 2060, 640, 16, False), (33, 1400, 1056, 16, False), (16, 49200, 128, 16, True)])
@pytest.mark.parametrize("fmt,with_zeros,odt", KINDS)
def test_tokens(m, n, k, tile, streamed, fmt, with_zeros, odt):
    require_gpu()
    p = rules.plan(m, n, k, 32, with_zeros)
    assert (p.tokens, p.streamed) == (tile, streamed)
    rng = np.random.default_rng(m)
    w, s, z = device_matrix(m, (), n, k, 32, "f32", with_zeros)
    x = bf16(rng.normal(size=(m, k)))[0]

    def product(x):
        out = torch.full((m, n), 5.0, dtype=odt, device="cuda")
        return b.fp8_w4_matvec(x, w, s, out, FMT[fmt], z)

    ref = product(x)
    order = torch.from_numpy(rng.permutation(m)).cuda()
    assert torch.equal(product(x[order]), ref[order])
    for kept in (0, m // 2, m - 1):
        other = bf16(rng.normal(size=(m, k)) * 100)[0]
        other[(kept + 1) % m] = float("nan")
        other[kept] = x[kept]
        assert torch.equal(product(other)[kept], ref[kept])


@pytest.mark.parametrize("P,E,n,k,tile,streamed", [
    (6, 50, 100, 1152, 1, False), (30, 32, 90, 1152, 4, False), (60, 64, 700, 256, 4, True),
    (100, 6, 200, 640, 16, False), (150, 9, 500, 640, 16, False), (200, 24, 2050, 256, 16, True)])
@pytest.mark.parametrize("fmt,with_zeros,odt", KINDS)
def test_pairs(P, E, n, k, tile, streamed, fmt, with_zeros, odt):
    require_gpu()
    p = rules.plan(P, n, k, 32, with_zeros, E)
    assert (p.tokens, p.streamed) == (tile, streamed)
    rng = np.random.default_rng(P)
    w, s, z = device_matrix(P, (E,), n, k, 32, "f32", with_zeros)
    x = bf16(rng.normal(size=(P, k)))[0]
    e = rng.integers(-1, E, P).astype(np.int32)
    e[rng.random(P) < 0.3] = e[0] = E - 1  # more than a tile of one expert

    def product(x, e):
        out = torch.full((P, n), 5.0, dtype=odt, device="cuda")
        return b.fp8_w4_matvec_experts(x, dev(e), w, s, out, FMT[fmt], z)

    ref = product(x, e)
    order = rng.permutation(P)
    assert torch.equal(product(x[torch.from_numpy(order).cuda()], e[order]), ref[torch.from_numpy(order).cuda()])
    for kept in (0, P // 2, P - 1):  # the others go elsewhere, with other values
        other, elsewhere = bf16(rng.normal(size=(P, k)) * 100)[0], rng.integers(-1, E, P).astype(np.int32)
        other[(kept + 1) % P] = float("nan")
        other[kept], elsewhere[kept] = x[kept], e[kept]
        assert torch.equal(product(other, elsewhere)[kept], ref[kept])
