"""The compiled way to the routing, combine and 4-bit calls: it makes the same
calls as the binding's own checks and leaves every unusual argument to them."""
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b

pytestmark = pytest.mark.gpu


def arguments():
    if not torch.cuda.is_available():
        pytest.fail("no GPU: this test needs one")
    torch.manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda")
    i = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.int32, device="cuda")
    e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    bf = torch.bfloat16
    codes = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda")
    return {
        "moe_route": [r(5, 16), 3, 1, r(16), 4, 2, 1, True, 2.5, e(5, 3, dt=torch.int32), e(5, 3)],
        "moe_route_backward": [r(5, 16).to(bf), i(0, 16, 5, 3), r(5, 3), e(5, 16, dt=bf), 0, False, 1.0],
        "moe_combine": [r(20, 64).to(bf), i(-1, 20, 5, 3), r(5, 3), e(5, 64, dt=bf)],
        "moe_combine_backward": [r(5, 64).to(bf), r(15, 64).to(bf), None, r(5, 3), e(15, 64, dt=bf), e(5, 3)],
        "w4_matvec": [r(3, 256).to(bf), codes(40, 128), r(40, 4), e(3, 40), 0, codes(40, 4)],
        "w4_matvec_experts": [r(3, 256).to(bf), i(-1, 5, 3, 2), codes(5, 24, 128), r(5, 24, 8).to(bf),
                              e(6, 24, dt=bf), 1, None]}


NAMES = ["moe_route", "moe_route_backward", "moe_combine", "moe_combine_backward", "w4_matvec", "w4_matvec_experts"]


class Sub(torch.Tensor):
    pass


@pytest.mark.parametrize("name", NAMES)
def test_same_results_as_the_bindings_own_checks(name):
    """With a stream given the binding makes the call itself; without one it is made directly."""
    b.lib()
    assert b._direct is not None
    results = []
    for stream in (None, torch.cuda.current_stream()):
        a = arguments()[name]
        if name == "moe_route":
            b.fp8_moe_route(a[0], a[1], a[2], a[3], *a[4:9], expert_idx=a[9], weights=a[10], stream=stream)
        else:
            getattr(b, "fp8_" + name)(*a, stream=stream)
        torch.cuda.synchronize()
        results.append([t for t in a if isinstance(t, torch.Tensor)])
    assert all(torch.equal(x, y) for x, y in zip(*results))
    assert getattr(b._direct, name)(*arguments()[name]) == b.FP8G_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_unusual_arguments_are_left_to_the_binding(name):
    b.lib()
    call = getattr(b._direct, name)
    good = arguments()[name]
    assert call(*good[:-1]) is None and call(*good, None) is None
    for at, v in enumerate(good):
        wrong = ["text", [1]]
        if isinstance(v, torch.Tensor):
            wide = torch.cat([v, v], -1)
            wrong += [None] if v.dim() > 1 and not (name == "moe_combine" and at in (1, 2)) and \
                not (name == "moe_combine_backward" and at == 5) and not (name == "w4_matvec" and at == 5) else []
            wrong += [v.cpu(), v.to(torch.float64), wide, torch.cat([v, v]), v.unsqueeze(0), v.as_subclass(Sub),
                      7, v[:0], wide[..., ::2] if v.dim() > 1 else wide[::2]]
            if v.dtype == torch.float32 and (name, at) not in (("w4_matvec", 2), ("w4_matvec", 3), ("moe_route", 0)):
                wrong.append(v.to(torch.bfloat16))
        elif isinstance(v, int) and not isinstance(v, bool):
            wrong += [1 << 40, 1.5]
        for x in wrong:
            a = list(good)
            a[at] = x
            if (name, at) in (("moe_route", 7), ("moe_route_backward", 5)):  # any truth value
                continue
            if name == "moe_combine" and at == 0 and isinstance(x, torch.Tensor) and x.shape[-1:] == v.shape[-1:] and \
                    x.is_contiguous() and type(x) is torch.Tensor and x.is_cuda and x.dtype == v.dtype:
                continue  # y may have any number of rows
            if name == "w4_matvec_experts" and at == 0 and getattr(x, "shape", ())[-1:] == v.shape[-1:] and \
                    len(x.shape) == 2 and len(x) == 6 and x.is_cuda and x.dtype == v.dtype:
                continue  # a row of x per pair
            if name == "w4_matvec_experts" and at == 1 and isinstance(x, torch.Tensor) and x.shape == (1, *v.shape):
                continue  # the pairs in any shape
            assert call(*a) != b.FP8G_OK, (name, at, x)  # None, or the library's refusal
    torch.cuda.synchronize()


def test_errors_of_the_library_are_raised():
    a = arguments()
    x = a["w4_matvec"]
    with pytest.raises(b.Fp8GemmError):
        b.fp8_w4_matvec(x[0], x[1], torch.ones(40, 16, device="cuda"), x[3])  # groups of 16
    r = a["moe_route"]
    with pytest.raises(b.Fp8GemmError):
        b.fp8_moe_route(r[0], 3, 1, expert_groups=5, topk_groups=1, expert_idx=r[9], weights=r[10])
