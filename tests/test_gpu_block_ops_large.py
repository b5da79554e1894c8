"""Norms, the dense epilogue and their gradients where offsets pass 32 bits and
where a workgroup takes many short rows.  A row's outputs do not depend on the
other rows, so the last rows of a large call are compared, bit for bit, with a
call on these rows alone (which runs the same kernels); sums over rows, of
gradients that are zero above them, with 64 bits.  Tolerances, with u = 2^-24: a
sum of N rows in FP32 is off by N u of the sum of absolute values."""
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from _gpu import require_gpu
from test_gpu_norm_residual import backward, case, check_gradients

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TAIL = 2000


def randn(*shape):
    t = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for at in range(0, shape[0], 1 << 15):
        t[at:at + (1 << 15)].normal_()
    return t


def test_norms_past_32_bit_offsets():
    require_gpu()
    torch.manual_seed(1)
    T, n = 300032, 7168
    assert T * n > 2 ** 31
    x, r = randn(T, n), randn(T, n)
    gate, pre, post = randn(n), randn(n), randn(n)
    kw = dict(pre_weight=pre, post_norm=True, post_weight=post, gate=gate, residual_scale=0.5)

    def forward(x, r):
        rows = x.shape[0]
        h, y = torch.empty_like(x), torch.empty_like(x)
        q = torch.empty(rows, n, dtype=torch.uint8, device="cuda")
        s = torch.empty(n // 128, rows, device="cuda")
        b.fp8_norm_residual(x, r, h, y, q, s, **kw)
        return h, y, q, s

    h, y, q, s = forward(x, r)
    h2, y2, q2, s2 = forward(x[-TAIL:], r[-TAIL:])
    assert torch.equal(h[-TAIL:], h2) and torch.equal(y[-TAIL:], y2) and torch.equal(q[-TAIL:], q2)
    assert torch.equal(s[:, -TAIL:], s2)
    del q, s, y

    gy = torch.zeros_like(x)
    gy[-TAIL:] = randn(TAIL, n)
    gh = torch.zeros_like(x)
    g_pre = torch.empty(n, device="cuda")
    gx, gr = torch.empty_like(x), torch.empty_like(x)
    b.fp8_norm_residual_backward(gh, gy, x, h, gx, gr, g_pre, **kw)
    gx2, gr2 = torch.empty_like(gx[-TAIL:]), torch.empty_like(gr[-TAIL:])
    b.fp8_norm_residual_backward(gh[-TAIL:], gy[-TAIL:], x[-TAIL:], h2, gx2, gr2, torch.empty_like(g_pre), **kw)
    assert torch.equal(gx[-TAIL:], gx2) and torch.equal(gr[-TAIL:], gr2)
    assert not gx[:1000].any() and not gr[:1000].any()
    hd, gd = h2.double(), gy[-TAIL:].double()
    terms = gd * hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert ((g_pre.double() - terms.sum(0)).abs() <= (TAIL + 200) * U * terms.abs().sum(0)).all()


def test_epilogue_past_32_bit_offsets():
    require_gpu()
    torch.manual_seed(2)
    m, n, k = 140000, 16384, 128
    assert m * n > 2 ** 31
    table = torch.tensor([c for c in range(256) if c & 127 < 126], dtype=torch.uint8, device="cuda")
    codes = lambda *shape: table[torch.randint(len(table), shape, device="cuda")]
    lhs, rhs = codes(m, k), codes(n, k)
    ls, rs = torch.rand(1, m, device="cuda") * 0.01, torch.rand(n // 128, 1, device="cuda") * 0.01
    bias = torch.randn(n, device="cuda")
    out = randn(m, n)
    residual = out[-TAIL:].clone()
    preact = torch.empty_like(out)
    kw = dict(bias=bias, activation=b.FP8G_ACT_GELU)
    b.fp8_gemm_nt_epilogue(lhs, ls, rhs, rs, out, residual=out, preact=preact, **kw)
    out2, preact2 = torch.empty_like(residual), torch.empty_like(residual)
    b.fp8_gemm_nt_epilogue(lhs[-TAIL:], ls[:, -TAIL:].contiguous(), rhs, rs, out2, residual=residual, preact=preact2, **kw)
    assert torch.equal(out[-TAIL:], out2) and torch.equal(preact[-TAIL:], preact2)

    grad = out  # zero but for the last rows
    grad[:-TAIL] = 0
    g_bias = torch.empty(n, device="cuda")
    z = preact2.double().requires_grad_()
    torch.nn.functional.gelu(z).sum().backward()
    terms = grad[-TAIL:].double() * z.grad
    size = grad[-TAIL:].double().abs().sum(0)
    grad2 = torch.empty_like(residual)
    b.fp8_epilogue_backward(grad[-TAIL:].clone(), preact2, b.FP8G_ACT_GELU, grad2)
    b.fp8_epilogue_backward(grad, preact, b.FP8G_ACT_GELU, preact, g_bias)  # in place
    assert torch.equal(preact[-TAIL:], grad2) and not preact[:1000].any()
    assert ((g_bias.double() - terms.sum(0)).abs() <= 2.0 ** -19 * size + (TAIL + 64) * U * terms.abs().sum(0)).all()


@pytest.mark.parametrize("T,n", [(9001, 128), (4999, 1536), (1030, 2048)])
@pytest.mark.parametrize("layer,gate,p_type", [(False, "one", "bf16"), (True, "row", "f32"), (True, None, "bf16")])
def test_gradients_of_many_short_rows(T, n, layer, gate, p_type):
    require_gpu()
    c = case(T, n, "bf16", "f32", p_type, True, gate, True, seed=T + n)
    g = torch.Generator().manual_seed(n)
    h = torch.randn(T, n, generator=g).cuda()
    gh, gy = torch.randn(T, n, generator=g).cuda(), torch.randn(T, n, generator=g).bfloat16().cuda()
    check_gradients(backward(c, gh, gy, h, True, layer), c, gh, gy, h, True, layer, 0.75)
