"""4-bit products over the whole range of their inputs: wherever a product is
defined and finite it is finite, and an infinity or a NaN gives what the
definition gives."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from oracle import moe_ops
from _gpu import dev, require_gpu
from test_gpu_moe_ops import Out, bf16
from test_gpu_w4 import DT, FMT, check, matrix

pytestmark = pytest.mark.gpu

KINDS = [("int4", "f32", False, "f32"), ("int4", "bf16", True, "f32"), ("e2m1", "f32", False, "f32"),
         ("int4", "f32", True, "bf16"), ("e2m1", "bf16", False, "bf16")]
# one token, tiles of 4, 8 and 16 tokens, of 16 and 32 rows, whole rows per wave of each
SHAPES = [(1, 70, 640), (3, 33, 1152), (8, 2049, 256), (13, 50, 384), (20, 4500, 256), (1, 33000, 256),
          (4, 25000, 256), (16, 49300, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", KINDS)
def test_sums_that_pass_the_range_before_their_scale(m, n, k, group, fmt, sdt, with_zeros, odt):
    """Activations of 1e37 to 1e38 with scales of about 0.01: a group's sum of
    unscaled codes passes FP32's range, the product does not."""
    require_gpu()
    rng = np.random.default_rng(m + n)
    tw, w, ts, s, tz, z = matrix(rng, (), n, k, group, sdt, with_zeros)
    big = np.where(np.arange(m) % 3 == 0, 2e37, 1.0)[:, None]
    tx, x = bf16((np.abs(rng.normal(size=(m, k))) + 0.5) * rng.choice([1, 1, 1, -1], (m, k)) * big)
    out = Out((m, n), DT[odt], 5)
    b.fp8_w4_matvec(tx, tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec(x, w, s, z, fmt == "e2m1")
    rows = np.arange(n) if n < 5000 else rng.permutation(n)[:5000]
    got, want, mag = out.numpy()[:, rows], want[:, rows], mag[:, rows]
    fits = np.abs(want) < (3.38e38 if odt == "bf16" else 3.4e38)
    assert fits.mean() > 0.5 and np.all(np.isfinite(got[fits]))
    check(got[fits], want[fits], mag[fits], k, odt)


@pytest.mark.parametrize("T,topk,E,n,k", [(1, 2, 40, 48, 640), (3, 2, 7, 40, 256), (40, 4, 3, 33, 256),
                                          (40, 8, 300, 130, 384), (64, 8, 100, 600, 128)])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", KINDS)
def test_experts_whose_sums_pass_the_range(T, topk, E, n, k, fmt, sdt, with_zeros, odt):
    require_gpu()
    rng = np.random.default_rng(T + n)
    e = rng.integers(-1, E, (T, topk)).astype(np.int32)
    e[0, 0] = E - 1
    tw, w, ts, s, tz, z = matrix(rng, (E,), n, k, 64, sdt, with_zeros)
    big = np.where(np.arange(T) % 3 == 0, 2e37, 1.0)[:, None]
    tx, x = bf16((np.abs(rng.normal(size=(T, k))) + 0.5) * big)
    out = Out((T * topk, n), DT[odt], 5)
    b.fp8_w4_matvec_experts(tx, dev(e), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec_experts(x, e, w, s, z, fmt == "e2m1")
    got = out.numpy()
    fits = np.abs(want) < (3.38e38 if odt == "bf16" else 3.4e38)
    assert fits.mean() > 0.5 and np.all(np.isfinite(got[fits]))
    check(got[fits], want[fits], mag[fits], k, odt)


@pytest.mark.parametrize("m,n,k", [(1, 40, 256), (4, 33000, 128), (16, 80, 512)])
@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
def test_infinities_by_the_definition(m, n, k, fmt):
    """An infinite activation times a value of its sign, of the other sign, of
    zero (NaN); two infinities that agree or cancel."""
    require_gpu()
    rng = np.random.default_rng(m)
    tw, w, ts, s, _, _ = matrix(rng, (), n, k, 32, "f32", False)
    tx, x = bf16(rng.normal(size=(m, k)))
    x[0, 7] = np.inf
    if m > 1:
        x[1, [40, 90]] = np.inf, -np.inf
        x[2, 3] = np.nan
    tx = bf16(x)[0]
    out = Out((m, n), torch.float32, 5)
    b.fp8_w4_matvec(tx, tw, ts, out.view, FMT[fmt])
    v, zero, scale = moe_ops.w4_parts(w, s, None, fmt == "e2m1")
    got = out.numpy()
    for i in range(min(m, 3)):
        with np.errstate(invalid="ignore"):
            want = (x[i].astype(np.float64) * ((v - zero) * scale)).sum(-1)
        special = ~np.isfinite(want)
        assert special.any() and np.array_equal(got[i][special], want[special], equal_nan=True)
        assert np.all(np.isfinite(got[i][~special]))


def test_finite_bound_of_unscaled_sums():
    """Both sides of where a group's unscaled sum passes the range: 128 columns
    of one value, code 9, zero 8 (9 x 128 x 2^117 < 2^128 <= 9 x 128 x 2^118)."""
    require_gpu()
    k, n = 128, 48
    w, s = np.full((n, k // 2), 0x99, np.uint8), np.full((n, 1), 2.0 ** -8, np.float32)
    for m in (1, 4, 16):
        for power in (110, 117, 118, 127):
            tx, x = bf16(np.full((m, k), 2.0 ** power))
            out = Out((m, n), torch.float32)
            b.fp8_w4_matvec(tx, dev(w), dev(s), out.view)
            assert np.array_equal(out.numpy(), np.full((m, n), 2.0 ** (power - 1), np.float32))


@pytest.mark.parametrize("m,n,k", [(1, 70, 2080), (3, 33, 1152), (8, 2060, 2560), (13, 50, 384), (20, 4500, 256),
                                   (4, 25000, 544), (16, 49300, 128)])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", KINDS)
def test_tokens_of_every_sort_in_a_tile(m, n, k, fmt, sdt, with_zeros, odt):
    """Ordinary ones, with a NaN at any place, with an infinity, and past the range before their scale."""
    require_gpu()
    rng = np.random.default_rng(m * k)
    tw, w, ts, s, tz, z = matrix(rng, (), n, k, 32, sdt, with_zeros)
    x = rng.normal(size=(m, k))
    sort = (np.arange(m) + 1) % 4  # 0 ordinary, 1 NaN, 2 large, 3 infinite
    x[sort == 2] = (np.abs(x[sort == 2]) + 0.5) * 2e37
    for i in np.nonzero(sort % 2)[0]:
        x[i, rng.integers(0, k)] = np.nan if sort[i] == 1 else -np.inf
    x[sort == 1, -1] = np.nan
    tx, x = bf16(x)
    out = Out((m, n), DT[odt], 5)
    b.fp8_w4_matvec(tx, tw, ts, out.view, FMT[fmt], tz)
    rows = np.arange(n) if n < 300 else np.unique(rng.integers(0, n, 300))
    got = out.numpy()[:, rows]
    v, zero, scale = moe_ops.w4_parts(w[rows], s[rows], None if z is None else z[rows], fmt == "e2m1")
    with np.errstate(invalid="ignore"):
        want = np.stack([(t * ((v - zero) * scale)).sum(-1) for t in x.astype(np.float64)])
    mag = np.abs(np.nan_to_num(x.astype(np.float64), posinf=0, neginf=0)) @ ((np.abs(v) + zero) * scale).T
    assert np.all(np.isnan(got[sort == 1]))
    special = ~np.isfinite(want)
    assert np.array_equal(got[special], want[special], equal_nan=True)
    fits = np.abs(want) < (3.38e38 if odt == "bf16" else 3.4e38)
    check(got[fits], want[fits], mag[fits], k, odt)
