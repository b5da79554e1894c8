"""More tokens than one launch has workgroups for."""
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from _gpu import require_gpu

pytestmark = pytest.mark.gpu


def test_combine_of_more_than_2_to_the_24_tokens():
    require_gpu()
    T, n = (1 << 24) + 5, 8
    w = (torch.arange(T, device="cuda") % 7 - 3).float().view(T, 1)
    y = (torch.arange(T * n, device="cuda") % 31).to(torch.bfloat16).view(T, n)  # products are exact in BF16
    want = (w * y.float()).to(torch.bfloat16)
    for dst in (None, torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)):
        rows = y if dst is None else y.flip(0)
        out = torch.full((T, n), 77.0, dtype=torch.bfloat16, device="cuda")
        b.fp8_moe_combine(rows, dst, w, out)
        assert torch.equal(out, want)
        gy, gw = torch.full_like(y, 77.0), torch.full_like(w, 77.0)
        b.fp8_moe_combine_backward(y, rows, dst, w, gy, gw)
        assert torch.equal(gy if dst is None else gy.flip(0), want)
        assert torch.equal(gw, y.float().square().sum(1, keepdim=True))  # whole numbers
