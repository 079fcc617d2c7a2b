"""The combination of the widest rows that are allowed, 2^31 - 8 columns, and its gradients: columns
are counted past 31 bits where a workgroup steps over the end. Integers that FP32 and BF16 hold,
so every sum is exact."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
N = 2 ** 31 - 8


def sparse(dev, *values):
    """[1, N], zero but for columns at the beginning, in the middle and at the end."""
    x = torch.zeros(1, N, dtype=BF16, device=dev)
    for at, v in zip((0, N // 2, N - 4096), values):
        x[0, at:at + 4096] = torch.arange(4096, device=dev) % 5 + v
    return x


def test_the_widest_rows(cuda_device):
    Y, w, at = sparse(cuda_device, 1, 2, 3), torch.tensor([[2.0]], device=cuda_device), torch.zeros(1, 1, dtype=I32, device=cuda_device)
    out = fg.moe_combine(Y, at, w)
    assert torch.equal(out, Y * 2)
    dO = sparse(cuda_device, 3, 1, 2)
    dY, dw = fg.moe_combine_backward(dO, Y, at, w, dY=out)
    assert torch.equal(dY, dO * 2)
    want = sum(int((dO[0, i:i + 4096].double() * Y[0, i:i + 4096].double()).sum()) for i in (0, N // 2, N - 4096))
    assert dw.tolist() == [[want]]
    assert fg.moe_combine_backward(dO, Y, at, w, rows=False)[1].tolist() == [[want]]
