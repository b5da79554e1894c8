"""With no bias, no activation and no residual the epilogue gives the plain
GEMM's bits, the sign of a zero among them: a sum of FP32 that underflows from
below is -0."""
import pytest
import torch

from fp8_block_scaled_04_amd import binding as b
from _gpu import require_gpu

pytestmark = pytest.mark.gpu


# every tile family, split over k (with a workspace) and not
@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (64, 2112, 7168), (128, 4096, 512), (96, 1544, 2048), (300, 512, 4096),
                                   (513, 4360, 256)])
def test_sums_that_underflow_keep_their_sign(m, n, k):
    require_gpu()
    lhs = torch.full((m, k), 0x01, dtype=torch.uint8, device="cuda")   # 2^-9
    rhs = torch.full((n, k), 0x01, dtype=torch.uint8, device="cuda")
    rhs[::2] = 0x81                                                    # -2^-9
    kg, tiny = k // 128, 2.0 ** -70  # scales of 2^-140 in all: a group's 128 products are -+2^-151, a quarter of FP32's least
    ls = torch.full((kg, (m + 3) // 4 * 4), tiny, device="cuda")
    rs = torch.full(((n + 127) // 128, kg), tiny, device="cuda")
    ws = torch.empty(max(16, b.fp8_gemm_workspace_bytes(m, n, k)), dtype=torch.uint8, device="cuda")
    want, out, pre = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    bits = lambda t: t.view(torch.int16)
    for workspace in (ws, None):
        b.fp8_gemm_nt(lhs, ls, rhs, rs, want, workspace=workspace)
        assert bool((bits(want) == -32768).any())  # the inputs are what they are meant to be
        b.fp8_gemm_nt_epilogue(lhs, ls, rhs, rs, out, preact=pre, workspace=workspace)
        assert torch.equal(bits(out), bits(want)) and torch.equal(bits(pre), bits(want))
        b.fp8_gemm_nt_epilogue(lhs, ls, rhs, rs, out, workspace=workspace)
        assert torch.equal(bits(out), bits(want))
