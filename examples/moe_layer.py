"""A mixture-of-experts layer on the library's calls, as a model would run it:

  decode    route -> the experts' products with 4-bit weights -> combine
  prefill   route -> grouped layout -> FP8 cast and scatter -> grouped GEMM -> combine
  training  the same forward pass, then the gradients of the combine and of the router's logits

python examples/moe_layer.py          (needs an MI355X and the built library)

Every result is compared with the same layer in plain FP32 torch; the largest
differences are printed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_04_amd as fp8  # noqa: E402

ROUTER = dict(score_func=fp8.FP8G_SIGMOID, expert_groups=4, topk_groups=2, group_score=fp8.FP8G_GROUP_TOP2,
              renormalize=True, scale=2.5)


def pack_int4(w, group=128):
    """FP32 weights [..][k] -> (codes [..][k / 2], BF16 scales, zero points [..][k / group]): 4 bits a weight, the even
    column of a pair in the low bits, each group's range spread over the codes 0..15."""
    parts = w.unflatten(-1, (-1, group))
    lo, hi = parts.amin(-1).clamp(max=0), parts.amax(-1).clamp(min=0)
    scales = ((hi - lo) / 15).clamp_min(1e-8).to(torch.bfloat16)
    zeros = (-lo / scales.float()).round().clamp(0, 15)
    codes = (parts / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scales, zeros.to(torch.uint8)


def unpack_int4(codes, scales, zeros):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (scales.shape[-1], -1))
    return ((c.float() - zeros.float()[..., None]) * scales.float()[..., None]).flatten(-2)


def difference(got, want):
    got, want = got.detach().float(), want.detach().float()
    return float((got - want).norm() / want.norm())


def decode(x, router, bias, up, down, topk):
    """x [T][h] BF16 -> [T][h]: two projections per routed expert, SwiGLU between them."""
    T, h = x.shape
    idx, weights = fp8.fp8_moe_route(x.float() @ router.t(), topk, bias=bias, **ROUTER)
    ff = down[0].shape[-1] * 2
    gate_up = torch.empty(T * topk, 2 * ff, dtype=torch.bfloat16, device=x.device)
    fp8.fp8_w4_matvec_experts(x, idx, up[0], up[1], gate_up, zeros=up[2])
    gate, value = gate_up.float().chunk(2, -1)
    act = (torch.nn.functional.silu(gate) * value).to(torch.bfloat16)
    y = torch.empty(T * topk, h, dtype=torch.bfloat16, device=x.device)
    fp8.fp8_w4_matvec_experts(act, idx, down[0], down[1], y, zeros=down[2])
    out = torch.empty(T, h, dtype=torch.bfloat16, device=x.device)
    fp8.fp8_moe_combine(y, None, weights, out)  # pair p in row p
    return out, idx, weights


def plain_decode(x, idx, weights, up, down):
    w_up, w_down = unpack_int4(*up), unpack_int4(*down)
    out = torch.zeros_like(x, dtype=torch.float32)
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e >= 0:
                gate, value = (w_up[e] @ x[t].float()).chunk(2)
                out[t] += weights[t, j] * (w_down[e] @ (torch.nn.functional.silu(gate) * value))
    return out


def prefill(x, logits, bias, w_codes, w_scales, topk):
    """x [T][h] BF16 through one FP8 projection per routed expert: (out, and what a backward pass needs)."""
    T, h = x.shape
    E, n = w_codes.shape[:2]
    idx, weights = fp8.fp8_moe_route(logits, topk, bias=bias, **ROUTER)
    _, _, dst, m_indices = fp8.fp8_moe_layout_contiguous(idx.view(-1), E)
    dst = dst.view(T, topk)
    ld = (T + 3) // 4 * 4
    q = torch.empty(T, h, dtype=torch.uint8, device=x.device)
    s = torch.empty(h // 128, ld, device=x.device)
    fp8.fp8_cast_per_token_group(x, q, s)
    M = m_indices.numel()
    rows = torch.zeros(M, h, dtype=torch.uint8, device=x.device)
    row_scales = torch.ones(h // 128, M, device=x.device)
    for j in range(topk):
        fp8.fp8_moe_scatter_rows(q, s, dst[:, j].contiguous(), rows, row_scales)
    y = torch.empty(M, n, dtype=torch.bfloat16, device=x.device)
    fp8.fp8_grouped_gemm_contiguous(rows, row_scales, w_codes, w_scales, y, m_indices)
    out = torch.empty(T, n, dtype=torch.bfloat16, device=x.device)
    fp8.fp8_moe_combine(y, dst, weights, out)
    return out, idx, weights, dst, y


def main():
    torch.manual_seed(0)
    dev, h, ff, E, topk = "cuda", 512, 256, 16, 4
    bias = torch.randint(-20, 21, (E,), device=dev) * 0.001
    router = torch.randn(E, h, device=dev) / h ** 0.5
    up = pack_int4(torch.randn(E, 2 * ff, h, device=dev) / h ** 0.5)
    down = pack_int4(torch.randn(E, h, ff, device=dev) / ff ** 0.5)
    worst = {}
    for T in (1, 7):
        x = torch.randn(T, h, device=dev).to(torch.bfloat16)
        out, idx, weights = decode(x, router, bias, up, down, topk)
        worst[f"decode, {T} tokens"] = difference(out, plain_decode(x, idx, weights, up, down))

    T, n = 300, 256
    x = torch.randn(T, h, device=dev).to(torch.bfloat16)
    w = torch.randn(E, n, h, device=dev) / h ** 0.5
    w_codes = torch.empty(E, n, h, dtype=torch.uint8, device=dev)
    w_scales = torch.empty(E, n // 128, h // 128, device=dev)
    for e in range(E):
        fp8.fp8_cast_per_block(w[e], w_codes[e], w_scales[e])
    logits = x.float() @ router.t()
    out, idx, weights, dst, y = prefill(x, logits, bias, w_codes, w_scales, topk)

    # the same with autograd, on the experts' rows that the FP8 product gave
    lp = logits.clone().requires_grad_(True)
    yp = y.float().requires_grad_(True)
    score = torch.sigmoid(lp).gather(1, idx.long())
    plain_weights = ROUTER["scale"] * score / score.sum(-1, keepdim=True)
    plain = (yp[dst.long()] * plain_weights[..., None]).sum(1)
    exact = torch.einsum("tjnh,th->tjn", w[idx.long()], x.float())
    worst["prefill, combine"] = difference(out, plain)
    worst["prefill, FP8 against FP32 weights"] = difference(out, (exact * plain_weights[..., None]).sum(1))

    grad_out = torch.randn(T, n, device=dev).to(torch.bfloat16)
    plain.backward(grad_out.float())
    grad_y = torch.zeros_like(y)  # padding rows have no gradient
    grad_weights = torch.empty_like(weights)
    fp8.fp8_moe_combine_backward(grad_out, y, dst, weights, grad_y, grad_weights)
    grad_logits = fp8.fp8_moe_route_backward(logits, idx, grad_weights, score_func=ROUTER["score_func"],
                                             renormalize=ROUTER["renormalize"], scale=ROUTER["scale"])
    worst["gradient of the experts' rows"] = difference(grad_y, yp.grad)
    worst["gradient of the logits"] = difference(grad_logits, lp.grad)
    for what, v in worst.items():
        print(f"{what}: relative difference {v:.2e}")
    return worst


if __name__ == "__main__":
    main()
