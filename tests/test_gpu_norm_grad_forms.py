"""Which of its two forms the norm's gradient takes: one launch, which leaves the workspace alone, or
two, which pass the weight's sums through it. Either way the sums are right (n 2^-24 of the terms'
magnitudes, as in the parity tests)."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,M,K,launches", [
    (FP32, 1024, 768, 2), (FP32, 1024, 1024, 2), (FP32, 1000, 1280, 2), (FP32, 900, 1536, 2),  # few columns, read twice: slower
    (FP32, 768, 1024, 1), (FP32, 1024, 512, 1), (FP32, 1024, 2048, 1), (FP32, 333, 2048, 1), (BF16, 1024, 1024, 1), (BF16, 256, 7168, 1),
    (FP32, 1100, 512, 2), (BF16, 1100, 1024, 2), (BF16, 300, 16384, 2)])
def test_launches(cuda_device, dtype, M, K, launches):
    if torch.cuda.get_device_properties(cuda_device).multi_processor_count != 256:
        pytest.skip("the sizes are for 256 compute units")
    g = synth.make_generator(60, cuda_device)
    dY, H = (torch.randn(M, K, generator=g, device=cuda_device).to(dtype) for _ in range(2))
    rstd, w = torch.ones(M, device=cuda_device), torch.ones(K, device=cuda_device)
    workspace = torch.full((fg.layer._fn("fp8_rmsnorm_backward_workspace_size")(M, K),), 0x5A, dtype=torch.uint8, device=cuda_device)
    _, dW = fg.rmsnorm_backward(dY, H, rstd, w, workspace=workspace)
    assert bool((workspace == 0x5A).all()) == (launches == 1)
    terms = dY.double() * H.double()
    assert bool(((dW.double() - terms.sum(dim=0)).abs() <= (M + 44) * 2.0 ** -24 * terms.abs().sum(dim=0)).all())
