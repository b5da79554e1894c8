"""Products with 4-bit weights on the GPU against the 64-bit oracle.

The tolerance follows from the definition: a group's sum adds products of a
BF16 value and a small integer or E2M1 value, which are exact in FP32, so k
additions of FP32 (2^-24 each, doubled where the matrix instruction rounds
toward zero), a zero point's product, one product per scale, and one rounding
of a BF16 output (2^-8)."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from oracle import moe_ops
from _gpu import dev, require_gpu
from test_gpu_moe_ops import Out, bf16, strided

pytestmark = pytest.mark.gpu


def matrix(rng, lead, n, k, group, sdt, with_zeros):
    codes = rng.integers(0, 256, (*lead, n, k // 2), dtype=np.uint8)
    s = np.exp(rng.normal(size=(*lead, n, k // group)) * 0.5).astype(np.float32) * 0.01
    ts, s = bf16(s) if sdt == "bf16" else (dev(s), s)
    z = rng.integers(0, 16, (*lead, n, k // group), dtype=np.uint8) if with_zeros else None
    return dev(codes), codes, ts, s, None if z is None else dev(z), z


def check(got, want, mag, k, odt):
    bound = mag * (2 * k + 16) * 2.0 ** -24 + (2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want) if odt == "bf16" else 0)
    worst = np.max(np.abs(got - want) - bound, initial=-1)
    assert np.all(np.abs(got - want) <= bound), f"worst excess {worst:.3g}"


TYPES = [  # format, scales, zero points, output
    ("int4", "bf16", False, "bf16"), ("int4", "f32", True, "f32"), ("int4", "bf16", True, "bf16"),
    ("e2m1", "bf16", False, "f32"), ("e2m1", "f32", False, "bf16")]
FMT = {"int4": b.FP8G_INT4, "e2m1": b.FP8G_E2M1}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SHAPES = [  # m, n, k
    (1, 1, 128), (1, 16, 128), (1, 17, 384), (2, 15, 640), (1, 100, 2048), (3, 64, 1152), (5, 33, 1280),
    (8, 48, 896), (16, 80, 2176), (17, 40, 1024), (31, 130, 256), (64, 70, 768), (65, 18, 512), (130, 9, 4224)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES)
def test_matvec(m, n, k, group, fmt, sdt, with_zeros, odt):
    require_gpu()
    rng = np.random.default_rng(m * 7 + n + k + group)
    tw, w, ts, s, tz, z = matrix(rng, (), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(m, k)))
    out = Out((m, n), DT[odt], 5)
    b.fp8_w4_matvec(strided(tx, 8 * (m % 3)), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec(x, w, s, z, fmt == "e2m1")
    check(out.numpy(), want, mag, k, odt)


@pytest.mark.parametrize("k,group", [(32, 32), (64, 32), (96, 32), (160, 32), (64, 64), (192, 64), (1056, 32), (2112, 64),
                                     (4128, 32)])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES)
def test_rows_that_end_inside_a_chunk(k, group, fmt, sdt, with_zeros, odt):
    """k of any number of groups: the last 128 columns may be part empty."""
    require_gpu()
    rng = np.random.default_rng(k)
    for m, n in ((1, 19), (6, 35)):
        tw, w, ts, s, tz, z = matrix(rng, (), n, k, group, sdt, with_zeros)
        tx, x = bf16(rng.normal(size=(m, k)))
        out = Out((m, n), DT[odt], 5)
        b.fp8_w4_matvec(tx, tw, ts, out.view, FMT[fmt], tz)
        want, mag = moe_ops.w4_matvec(x, w, s, z, fmt == "e2m1")
        check(out.numpy(), want, mag, k, odt)


def test_every_code_is_decoded():
    """Each of the 16 codes at every place of its dword, alone in its row,
    for every zero point: exact values."""
    require_gpu()
    k = 128
    for fmt, zeros in [("e2m1", [None]), ("int4", [None, 0, 1, 7, 8, 15, 200])]:
        for zero in zeros:
            codes = np.full((16 * 16, k), 0 if fmt == "e2m1" else (8 if zero is None else min(zero, 15)), np.uint8)
            for c in range(16):
                for p in range(16):
                    codes[c * 16 + p, p * 8 + p % 8] = c
            packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
            s = np.full((256, 1), 0.25, np.float32)
            z = None if zero is None else np.full((256, 1), zero, np.uint8)
            x = bf16(np.arange(1, k + 1)[None] * 1.0)
            out = Out((1, 256), torch.float32, 5)
            b.fp8_w4_matvec(x[0], dev(packed), dev(s), out.view, FMT[fmt], None if z is None else dev(z))
            want, _ = moe_ops.w4_matvec(x[1], packed, s, z, fmt == "e2m1")
            assert np.array_equal(out.numpy(), want), (fmt, zero)


def test_infinities_and_nan_stay_in_their_rows():
    """A token with an infinity or NaN spoils its own output row only, a
    matrix row with such a scale its own column only."""
    require_gpu()
    rng = np.random.default_rng(2)
    for m in (3, 20):
        tw, w, ts, s, _, _ = matrix(rng, (), 40, 512, 128, "f32", False)
        tx, x = bf16(rng.normal(size=(m, 512)))
        tx[1, 130], tx[2, 7] = float("inf"), float("nan")
        ts[5, 2] = float("nan")
        out = Out((m, 40), torch.float32)
        b.fp8_w4_matvec(tx, tw, ts, out.view)
        got = out.numpy()
        want, mag = moe_ops.w4_matvec(x, w, s)
        rows = [i for i in range(m) if i not in (1, 2)]
        cols = [j for j in range(40) if j != 5]
        check(got[np.ix_(rows, cols)], want[np.ix_(rows, cols)], mag[np.ix_(rows, cols)], 512, "f32")
        assert np.all(np.isnan(got[2])) and np.all(np.isnan(got[:, 5])) and not np.any(np.isfinite(got[1]))


EXPERTS = [  # T, topk, E, n, k, per pair
    (1, 1, 1, 16, 128, False), (1, 8, 64, 40, 512, False), (1, 8, 16, 24, 256, True), (3, 2, 4, 17, 384, False),
    (5, 6, 7, 33, 640, True), (40, 4, 3, 20, 256, False), (64, 8, 16, 48, 512, True), (200, 2, 5, 16, 128, False),
    (33, 3, 300, 16, 256, True)]


@pytest.mark.parametrize("T,topk,E,n,k,per_pair", EXPERTS)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES)
def test_experts(T, topk, E, n, k, per_pair, group, fmt, sdt, with_zeros, odt):
    require_gpu()
    rng = np.random.default_rng(T + E)
    e = rng.integers(0, E, (T, topk)).astype(np.int32)  # a token may name an expert twice
    if T > 2:
        e[rng.random((T, topk)) < 0.1] = rng.choice([-1, E, E + 9])
        e[1] = -1
    tw, w, ts, s, tz, z = matrix(rng, (E,), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(T * topk if per_pair else T, k)))
    out = Out((T * topk, n), DT[odt], 5)
    b.fp8_w4_matvec_experts(strided(tx, 8 * (T % 2)), dev(e), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec_experts(x, e, w, s, z, fmt == "e2m1")
    got = out.numpy()
    check(got, want, mag, k, odt)
    assert np.all(got[(e.reshape(-1) < 0) | (e.reshape(-1) >= E)] == 0)


STREAMS = [  # m, n, k: enough rows that no wave splits k
    (1, 32768, 128), (1, 40001, 320), (3, 33000, 256), (4, 32769, 1024), (5, 65536, 128), (16, 70007, 384),
    (19, 66000, 160), (1, 300000, 64)]


@pytest.mark.parametrize("m,n,k", STREAMS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES)
def test_matvec_of_many_rows(m, n, k, group, fmt, sdt, with_zeros, odt):
    require_gpu()
    k = k // group * group or group
    rng = np.random.default_rng(m + n + k)
    tw, w, ts, s, tz, z = matrix(rng, (), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(m, k)))
    out = Out((m, n), DT[odt], 5)
    b.fp8_w4_matvec(strided(tx, 8 * (m % 2)), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec(x, w, s, z, fmt == "e2m1")
    check(out.numpy(), want, mag, k, odt)


@pytest.mark.parametrize("T,topk,E,n,k,per_pair", [
    (1, 8, 64, 4100, 128, False), (2, 5, 40, 3500, 256, True), (40, 8, 300, 130, 384, False), (64, 8, 128, 270, 512, True),
    (30, 4, 500, 80, 1024, False), (900, 2, 9, 4000, 64, False), (7, 3, 60, 8200, 96, True)])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES)
def test_experts_of_many_rows(T, topk, E, n, k, per_pair, group, fmt, sdt, with_zeros, odt):
    require_gpu()
    k = k // group * group
    rng = np.random.default_rng(T + E + n)
    e = rng.integers(0, E, (T, topk)).astype(np.int32)
    if T > 2:
        e[rng.random((T, topk)) < 0.1] = rng.choice([-1, E, E + 9])
        e[1] = -1
    tw, w, ts, s, tz, z = matrix(rng, (E,), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(T * topk if per_pair else T, k)))
    out = Out((T * topk, n), DT[odt], 5)
    b.fp8_w4_matvec_experts(tx, dev(e), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec_experts(x, e, w, s, z, fmt == "e2m1")
    got = out.numpy()
    check(got, want, mag, k, odt)
    assert np.all(got[(e.reshape(-1) < 0) | (e.reshape(-1) >= E)] == 0)


@pytest.mark.parametrize("m,n,k", [
    (1, 4096, 1152), (4, 4097, 1152), (1, 12288, 1056), (3, 12289, 1152), (1, 24560, 1056), (2, 24561, 1152),
    (16, 4096, 1152), (9, 4097, 1152), (17, 2048, 2176), (33, 1400, 2176), (16, 8192, 1056), (7, 8193, 1152),
    (5, 2111, 1056), (8, 4096, 1152),
    (8, 4097, 1152), (16, 2048, 1056), (7, 3000, 640), (30, 1000, 2176), (6, 2049, 384), (11, 2033, 160),
    (16, 24576, 640), (8, 24577, 640), (12, 49120, 320), (16, 49121, 320), (1, 560000, 64), (16, 1050000, 32)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES[1:3] + TYPES[4:])
def test_matvec_around_each_split(m, n, k, group, fmt, sdt, with_zeros, odt):
    """Numbers of rows on both sides of where fewer waves share them, and where a wave takes several sets of them."""
    require_gpu()
    k = k // group * group or group
    n = min(n, (1 << 25) // k)
    rng = np.random.default_rng(m + n + k)
    tw, w, ts, s, tz, z = matrix(rng, (), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(m, k)))
    out = Out((m, n), DT[odt], 5)
    b.fp8_w4_matvec(strided(tx, 8 * (m % 2)), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec(x, w, s, z, fmt == "e2m1")
    check(out.numpy(), want, mag, k, odt)


@pytest.mark.parametrize("T,topk,E,n,k,per_pair", [
    (500, 1, 500, 1040, 64, False), (400, 1, 300, 3700, 64, True), (4, 2, 9, 1000, 1056, False),
    (5, 2, 8, 456, 1152, True), (1, 3, 40, 4096, 640, False), (2, 3, 6, 4097, 640, True)])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("fmt,sdt,with_zeros,odt", TYPES[1:3] + TYPES[4:])
def test_experts_around_each_split(T, topk, E, n, k, per_pair, group, fmt, sdt, with_zeros, odt):
    require_gpu()
    k = k // group * group
    rng = np.random.default_rng(T + E + n)
    e = rng.integers(0, E, (T, topk)).astype(np.int32)
    tw, w, ts, s, tz, z = matrix(rng, (E,), n, k, group, sdt, with_zeros)
    tx, x = bf16(rng.normal(size=(T * topk if per_pair else T, k)))
    out = Out((T * topk, n), DT[odt], 5)
    b.fp8_w4_matvec_experts(tx, dev(e), tw, ts, out.view, FMT[fmt], tz)
    want, mag = moe_ops.w4_matvec_experts(x, e, w, s, z, fmt == "e2m1")
    check(out.numpy(), want, mag, k, odt)


@pytest.mark.parametrize("T,topk,E,n,k", [
    (700, 1, 70, 100, 256), (40, 8, 200, 60, 128), (9000, 1, 70, 33, 64), (32768, 2, 90, 20, 32),
    (64, 8, 100, 4500, 64), (16, 4, 64, 50, 512)])
@pytest.mark.parametrize("hot", [(0,), (69, 3), (63, 64, -1)])
def test_experts_of_a_few_hot_ones(T, topk, E, n, k, hot):
    """Most pairs with one to three experts: tiles of one expert by the dozen, other experts with one pair or none."""
    require_gpu()
    rng = np.random.default_rng(T + E)
    hot = [h if h < E else E - 1 for h in hot]
    e = rng.choice(np.int32(hot), (T, topk))
    e[rng.random((T, topk)) < 0.1] = rng.integers(-1, E)
    tw, w, ts, s, tz, z = matrix(rng, (E,), n, k, 32, "bf16", True)
    tx, x = bf16(rng.normal(size=(T, k)))
    out = Out((T * topk, n), torch.float32, 5)
    b.fp8_w4_matvec_experts(tx, dev(e.astype(np.int32)), tw, ts, out.view, zeros=tz)
    want, mag = moe_ops.w4_matvec_experts(x, e, w, s, z)
    got = out.numpy()
    check(got, want, mag, k, "f32")
    assert np.all(got[e.reshape(-1) < 0] == 0)


def test_streamed_matrices_past_32_bits():
    """Experts past 2^32 bytes, with enough pairs for whole rows per wave."""
    require_gpu()
    rng = np.random.default_rng(7)
    E, n, k = 140, 16384, 4096
    w = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, n, k // 64, device="cuda")
    for g in (0, 139):
        w[g] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
        s[g] = 0.01
    tx, x = bf16(rng.normal(size=(2, k)))
    out = torch.empty(4, n, device="cuda")
    b.fp8_w4_matvec_experts(tx, dev(np.int32([[139, 0], [0, 139]])), w, s, out)
    for p, g in enumerate((139, 0, 0, 139)):
        rows = [0, 17, 4095, n - 1]
        want, mag = moe_ops.w4_matvec(x[p // 2:p // 2 + 1], w[g][rows].cpu().numpy(), s[g][rows].cpu().numpy())
        check(out[p][rows].cpu().numpy()[None], want, mag, k, "f32")


def test_matrices_past_32_bits():
    """Experts whose codes start past 2^32 bytes."""
    require_gpu()
    rng = np.random.default_rng(6)
    E, n, k = 70, 8192, 16384
    w = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, n, k // 128, device="cuda")
    for g in (0, 68):
        w[g] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
        s[g] = 0.01
    tx, x = bf16(rng.normal(size=(1, k)))
    e = dev(np.int32([[68, 0]]))
    out = torch.empty(2, n, device="cuda")
    b.fp8_w4_matvec_experts(tx, e, w, s, out)
    for p, g in enumerate((68, 0)):
        rows = [0, 1, 4095, n - 1]
        want, mag = moe_ops.w4_matvec(x, w[g][rows].cpu().numpy(), s[g][rows].cpu().numpy())
        check(out[p][rows].cpu().numpy()[None], want, mag, k, "f32")


def test_results_do_not_depend_on_the_batch_or_the_run():
    """Same bits on every run, on another stream and in graph replays."""
    require_gpu()
    rng = np.random.default_rng(9)
    tw, _, ts, _, tz, _ = matrix(rng, (4,), 200, 1024, 64, "bf16", True)
    tx, _ = bf16(rng.normal(size=(6, 1024)))
    e = dev(rng.integers(0, 4, (6, 2)).astype(np.int32))
    out, one = (torch.empty(n, 200, dtype=torch.bfloat16, device="cuda") for n in (12, 6))

    def step(stream=None):
        b.fp8_w4_matvec_experts(tx, e, tw, ts, out, zeros=tz, stream=stream)
        b.fp8_w4_matvec(tx, tw[1], ts[1], one, zeros=tz[1], stream=stream)

    step()
    torch.cuda.synchronize()
    ref = out.clone(), one.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_(), one.zero_()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(one, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        out.zero_(), one.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(one, ref[1])
        step()


def test_empty_products():
    require_gpu()
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    b.fp8_w4_matvec(h(0, 128), u(8, 64), h(8, 1), h(0, 8))
    b.fp8_w4_matvec(h(2, 128), u(0, 64), h(0, 1), h(2, 0))
    out = torch.full((2, 8), 3.0, device="cuda")
    b.fp8_w4_matvec(h(2, 0), u(8, 0), h(8, 0), out)  # an empty sum
    assert float(out.abs().sum()) == 0
    b.fp8_w4_matvec_experts(h(0, 128), torch.zeros(0, 4, dtype=torch.int32, device="cuda"), u(3, 8, 64), h(3, 8, 1),
                            h(0, 8))


def test_binding_refuses_wrong_tensors():
    require_gpu()
    f = lambda *s: torch.zeros(s, device="cuda")
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for bad, err in [
            (lambda: b.fp8_w4_matvec(f(2, 128), u(8, 64), h(8, 1), h(2, 8)), TypeError),
            (lambda: b.fp8_w4_matvec(h(2, 128), h(8, 64), h(8, 1), h(2, 8)), TypeError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 32), h(8, 1), h(2, 8)), ValueError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(7, 1), h(2, 8)), ValueError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 3), h(2, 8)), ValueError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), u(8, 1), h(2, 8)), TypeError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 1), h(2, 7)), ValueError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 1), h(2, 8), zeros=u(8, 2)), ValueError),
            (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 1), h(2, 8), zeros=h(8, 1)), TypeError),
            (lambda: b.fp8_w4_matvec(h(128, 2).t(), u(8, 64), h(8, 1), h(2, 8)), ValueError),
            (lambda: b.fp8_w4_matvec_experts(h(2, 128), i(3), u(4, 8, 64), h(4, 8, 1), h(3, 8)), ValueError),
            (lambda: b.fp8_w4_matvec_experts(h(2, 128), i(2), u(4, 8, 64), h(3, 8, 1), h(2, 8)), ValueError),
            (lambda: b.fp8_w4_matvec_experts(h(2, 128), i(2), u(8, 64), h(8, 1), h(2, 8)), ValueError)]:
        with pytest.raises(err):
            bad()
    for bad in (lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 8), h(2, 8)),  # groups of 16
                lambda: b.fp8_w4_matvec(h(2, 256), u(8, 128), h(8, 1), h(2, 8)),  # groups of 256
                lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 1), h(2, 8), w_format=2),
                lambda: b.fp8_w4_matvec(h(2, 132)[:, :128], u(8, 64), h(8, 1), h(2, 8)),  # stride
                lambda: b.fp8_w4_matvec(h(2, 136)[:, 4:132], u(8, 64), h(8, 1), h(2, 8)),  # alignment
                lambda: b.fp8_w4_matvec(h(2, 128), u(8, 64), h(8, 1), h(2, 8), b.FP8G_E2M1, u(8, 1))):
        with pytest.raises(b.Fp8GemmError):
            bad()
