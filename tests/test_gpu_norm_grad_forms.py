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


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,K", [(1, 256), (37, 2048), (333, 1152), (1024, 1024), (1024, 4096), (1500, 640), (300, 16384)])
def test_the_order_of_the_sums_is_fixed(cuda_device, dtype, M, K):
    """dX apart, in dY's, dH's or H's place, or in rows that alternate with theirs: always the same
    dX; and the same dW wherever dX meets dY or H, and wherever it meets neither."""
    g = synth.make_generator(61, cuda_device)
    dY, H, dH = (torch.randn(M, K, generator=g, device=cuda_device).to(dtype) for _ in range(3))
    w = torch.randn(K, generator=g, device=cuda_device)
    rstd = torch.rand(M, generator=g, device=cuda_device) + 0.5
    met = {}
    for extra in (dH, None):
        dX, dW = fg.rmsnorm_backward(dY, H, rstd, w, dH=extra)
        wide = torch.empty(M, 2 * K, dtype=dtype, device=cuda_device)
        for shared in (0, 1, 2) if extra is not None else (0, 1):
            for view in (None, wide[:, K:]):  # the shared input's own rows, or the gaps between them
                given = [dY, H, extra]
                own = given[shared].clone() if view is None else wide[:, :K].copy_(given[shared])
                given[shared] = own
                x, s = fg.rmsnorm_backward(given[0], given[1], rstd, w, dH=given[2], dX=own if view is None else view)
                assert torch.equal(x, dX)
                first = dW if shared == 2 else met.setdefault(extra is None, s)
                assert torch.equal(s, first)
