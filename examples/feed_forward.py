"""The feed-forward block of a model on the library's calls, as training and decoding would run it:

  dense     norm with gate and residual -> FP8 codes -> up projection (bias, GELU) -> FP8 cast -> down projection
            added to the residual; and the gradients that stand around the products
  experts   routing -> the whole mixture-of-experts layer in one call -> norm with the residual, for a few tokens, with
            the FP8 matrices that the grouped GEMMs of a prefill take

python examples/feed_forward.py          (needs an MI355X and the built library)

Every result is compared with the same block in plain FP32 torch; the largest differences are printed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_04_amd as fp8  # noqa: E402

BF16 = torch.bfloat16


def rms(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w


def scales_for(rows, k, device):
    return torch.empty(k // 128, (rows + 3) // 4 * 4, device=device)


def block_cast(w):
    """FP32 [..][n][k] -> (E4M3 codes, a scale per 128 x 128 block)."""
    flat = w.reshape(-1, *w.shape[-2:])
    q = torch.empty(flat.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty(flat.shape[0], (w.shape[-2] + 127) // 128, w.shape[-1] // 128, device=w.device)
    for e in range(flat.shape[0]):
        fp8.fp8_cast_per_block(flat[e], q[e], s[e])
    return q.view(w.shape), s.view(*w.shape[:-2], *s.shape[-2:])


def values(q, s):
    """FP32 values of a block cast."""
    s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)
    return q.view(torch.float8_e4m3fn).float() * s


def difference(got, want):
    got, want = got.detach().float(), want.detach().float()
    return float((got - want).norm() / want.norm())


def dense_block(x, residual, p):
    """x: the attention's output, residual: the stream [T][h], BF16 -> (the stream after the block, what a backward
    pass needs)."""
    T, h = x.shape
    ff = p["up"].shape[0]
    stream = torch.empty_like(residual)
    q = torch.empty(T, h, dtype=torch.uint8, device=x.device)
    s = scales_for(T, h, x.device)
    fp8.fp8_norm_residual(x, residual, stream, q=q, q_scales=s, pre_weight=p["pre"], post_norm=True,
                          post_weight=p["post"], gate=p["gate"])
    act, z = torch.empty(T, ff, dtype=BF16, device=x.device), torch.empty(T, ff, dtype=BF16, device=x.device)
    work = torch.empty(max(4, fp8.fp8_gemm_workspace_bytes(T, ff, h), fp8.fp8_gemm_workspace_bytes(T, h, ff)),
                       dtype=torch.uint8, device=x.device)
    fp8.fp8_gemm_nt_epilogue(q, s, p["up"], p["up_scales"], act, bias=p["bias"], activation=fp8.FP8G_ACT_GELU_TANH,
                             preact=z, workspace=work)
    aq = torch.empty(T, ff, dtype=torch.uint8, device=x.device)
    asc = scales_for(T, ff, x.device)
    fp8.fp8_cast_per_token_group(act, aq, asc)
    out = torch.empty_like(stream)
    fp8.fp8_gemm_nt_epilogue(aq, asc, p["down"], p["down_scales"], out, residual=stream, workspace=work)
    return out, stream, z


def dense_block_backward(grad_out, x, stream, z, p):
    """The gradients of x, the residual and the parameters around the products, for a gradient of the block's output.
    The products' own gradients go through plain matrix products here."""
    grad_act = (grad_out.float() @ values(p["down"], p["down_scales"])).to(BF16)
    grad_z, grad_bias = torch.empty_like(z), torch.empty(z.shape[1], device=z.device)
    fp8.fp8_epilogue_backward(grad_act, z, fp8.FP8G_ACT_GELU_TANH, grad_z, grad_bias)
    grad_y = (grad_z.float() @ values(p["up"], p["up_scales"])).to(BF16)
    grad_x, grad_residual = torch.empty_like(x), torch.empty_like(x)
    h = x.shape[1]
    grad_pre, grad_post, grad_gate = (torch.empty(h, device=x.device) for _ in range(3))
    fp8.fp8_norm_residual_backward(grad_out, grad_y, x, stream, grad_x, grad_residual, grad_pre, grad_post, grad_gate,
                                   pre_weight=p["pre"], post_norm=True, post_weight=p["post"], gate=p["gate"])
    return dict(x=grad_x, residual=grad_residual, bias=grad_bias, pre=grad_pre, post=grad_post, gate=grad_gate)


def plain_dense(x, residual, p):
    """The same block in FP32, the weights' codes decoded, without the activations' casts."""
    stream = residual + p["gate"] * rms(x, p["post"])
    act = torch.nn.functional.gelu(rms(stream, p["pre"]) @ values(p["up"], p["up_scales"]).t() + p["bias"],
                                   approximate="tanh")
    return stream + act @ values(p["down"], p["down_scales"]).t()


def experts_block(x, residual, router, p, topk):
    """A decoding step: the routed experts' feed-forward networks of a few tokens, then the next block's input."""
    idx, weights = fp8.fp8_moe_route(x.float() @ router.t(), topk, renormalize=True)
    y = torch.empty_like(x)
    fp8.fp8_moe_few_tokens(x, idx, weights, p["up"], p["up_scales"], p["down"], p["down_scales"], y)
    stream, nxt = torch.empty_like(residual), torch.empty_like(x)
    fp8.fp8_norm_residual(y, residual, stream, nxt, pre_weight=p["pre"])
    return stream, nxt, idx, weights


def plain_experts(x, residual, idx, weights, p):
    out = residual.float().clone()
    up, down = values(p["up"], p["up_scales"]), values(p["down"], p["down_scales"])
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            gate, value = (up[e] @ x[t].float()).chunk(2)
            out[t] += weights[t, j] * (down[e] @ (torch.nn.functional.silu(gate) * value))
    return out, rms(out, p["pre"].float())


def main():
    torch.manual_seed(0)
    dev, T, h, ff = "cuda", 300, 512, 1024
    randn = lambda *s: torch.randn(*s, device=dev)
    p = {"pre": (1 + 0.1 * randn(h)), "post": (1 + 0.1 * randn(h)), "gate": (0.5 + 0.1 * randn(h)), "bias": 0.1 * randn(ff)}
    p["up"], p["up_scales"] = block_cast(randn(ff, h) / h ** 0.5)
    p["down"], p["down_scales"] = block_cast(randn(h, ff) / ff ** 0.5)
    x, residual = randn(T, h).to(BF16), (2 * randn(T, h)).to(BF16)
    out, stream, z = dense_block(x, residual, p)
    leaves = {k: v.float().clone().requires_grad_(True) for k, v in
              dict(x=x, residual=residual, pre=p["pre"], post=p["post"], gate=p["gate"], bias=p["bias"]).items()}
    plain = plain_dense(leaves["x"], leaves["residual"], {**p, **leaves})
    worst = {"dense block": difference(out, plain)}
    grad_out = randn(T, h).to(BF16)
    grads = dense_block_backward(grad_out, x, stream, z, p)
    plain.backward(grad_out.float())
    for name, g in grads.items():
        worst[f"gradient of {name}"] = difference(g, leaves[name].grad)

    E, topk, inter = 16, 4, 384
    p["up"], p["up_scales"] = block_cast(randn(E, 2 * inter, h) / h ** 0.5)
    p["down"], p["down_scales"] = block_cast(randn(E, h, inter) / inter ** 0.5)
    router = randn(E, h) / h ** 0.5
    for T in (1, 7, 40):
        x, residual = randn(T, h).to(BF16), randn(T, h).to(BF16)
        stream, nxt, idx, weights = experts_block(x, residual, router, p, topk)
        want, want_next = plain_experts(x, residual, idx, weights, p)
        worst[f"experts, {T} tokens"] = difference(stream, want)
        worst[f"experts, {T} tokens, the next block's input"] = difference(nxt, want_next)
    for what, v in worst.items():
        print(f"{what}: relative difference {v:.2e}")
    return worst


if __name__ == "__main__":
    main()
