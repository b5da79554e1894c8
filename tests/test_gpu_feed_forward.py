"""The example of a feed-forward block: the norms, the products with their
epilogues, the expert layer and the gradients, one after another as a model runs
them, against plain torch."""
import importlib.util
import os

import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu
EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")


def test_example_block():
    require_gpu()
    spec = importlib.util.spec_from_file_location("feed_forward", EXAMPLE)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    worst = block.main()
    # The activations are cast to E4M3 twice on the way: steps of 2^-4 of a value, at most half of one off, in the branch
    # that is added to a stream twice its size.  The gradients are taken where those casts left z.
    assert worst["dense block"] < 2.0 ** -5
    for name in ("x", "residual", "bias", "pre", "post", "gate"):
        assert worst[f"gradient of {name}"] < 2.0 ** -4, name
    # BF16 outputs (2^-8 at most) of BF16 inputs, one after another
    for T in (1, 7, 40):
        assert worst[f"experts, {T} tokens"] < 2.0 ** -8
        assert worst[f"experts, {T} tokens, the next block's input"] < 2.0 ** -7


def test_without_the_compiled_module(monkeypatch):
    """The same calls through ctypes: the same bits, for outputs and gradients."""
    import torch

    from fp8_block_scaled_04_amd import binding as b

    require_gpu()
    g = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    f32 = lambda *s: torch.randn(*s, generator=g).cuda()
    codes = lambda *s: torch.randn(*s, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    x, r, gy, gate, w = bf(40, 256), f32(40, 256), bf(40, 256), f32(256), f32(256)
    lhs, rhs, bias = codes(40, 256), codes(512, 256), bf(512)
    ones = lambda *s: torch.ones(*s, device="cuda")
    idx = torch.randint(-1, 4, (40, 2), generator=g, dtype=torch.int32).cuda()
    up, down, weights = codes(4, 256, 256), codes(4, 256, 128), torch.rand(40, 2, generator=g).cuda()

    def run():
        e = lambda *s, dtype=torch.bfloat16: torch.full(s, 3, device="cuda").to(dtype)
        h, y, q, s = e(40, 256, dtype=torch.float32), e(40, 256), e(40, 256, dtype=torch.uint8), ones(2, 40)
        b.fp8_norm_residual(x, r, h, y, q, s, pre_weight=w, post_norm=True, post_weight=w, gate=gate, residual_scale=0.5,
                            kind=b.FP8G_NORM_LAYER, eps=1e-5)
        grads = e(40, 256), e(40, 256, dtype=torch.float32), *(e(256, dtype=torch.float32) for _ in range(3))
        b.fp8_norm_residual_backward(h, gy, x, h, *grads, pre_weight=w, post_norm=True, post_weight=w, gate=gate,
                                     residual_scale=0.5, kind=b.FP8G_NORM_LAYER, eps=1e-5)
        out, z, gz, gb = e(40, 512), e(40, 512), e(40, 512), e(512, dtype=torch.float32)
        b.fp8_gemm_nt_epilogue(lhs, ones(2, 40), rhs, ones(4, 2), out, bias=bias, activation=b.FP8G_ACT_SILU, preact=z,
                               residual=bias.expand(40, 512).contiguous())
        b.fp8_epilogue_backward(out, z, b.FP8G_ACT_GELU, gz, gb)
        moe = e(40, 256)
        b.fp8_moe_few_tokens(x, idx, weights, up, ones(4, 2, 2), down, ones(4, 2, 1), moe, activation=b.FP8G_ACT_RELU)
        return h, y, q, s, *grads, out, z, gz, gb, moe

    first = run()
    assert b._direct is not None
    monkeypatch.setattr(b, "_direct", None)
    assert all(torch.equal(u, v) for u, v in zip(first, run()))
