"""Calls at the edges of what the layer operators take."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("M", [1, 3, 6, 129])
def test_scales_of_one_block_row(cuda_device, M):
    """The first M columns of a wider buffer, as with more block rows."""
    g = synth.make_generator(2, cuda_device)
    for K in (128, 256):
        X, w = torch.randn(M, K, generator=g, device=cuda_device).to(BF16), torch.ones(K, device=cuda_device)
        want = fg.rmsnorm_quantize_1x128(X, w)
        wide = torch.full((K // 128, fg.scale_ld(M)), -7.0, device=cuda_device)
        sa = fg.rmsnorm_quantize_1x128(X, w, sa=wide[:, :M])[1]
        assert torch.equal(sa, want[1][:, :M]) and bool((wide[:, M:] == -7).all())
