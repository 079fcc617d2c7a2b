"""Calls at the edges of what the layer operators take."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from test_gpu_paged_append import table_of

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


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


def test_a_table_without_pages(cuda_device):
    """Nothing is stored and nothing is seen; queries turn by their slots all the same."""
    dev = cuda_device
    cache = fg.make_paged_kv_cache(2, 2, 16, 64, device=dev)
    before = [t.clone() for t in cache]
    g = synth.make_generator(1, dev)
    q, k, v = (torch.randn(5, h, 64, generator=g, device=dev).to(BF16) for h in (4, 2, 2))
    lens, cu = (torch.tensor(x, dtype=I32, device=dev) for x in ([3, 9], [0, 3, 5]))
    table, rot = torch.empty(2, 0, dtype=I32, device=dev), table_of(16, 32, dev)
    got = fg.rope_append_paged_kv(q, k, v, rot, cache, table, lens, cu)
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    other = fg.make_paged_kv_cache(2, 2, 16, 64, device=dev)
    want = fg.rope_append_paged_kv(q, k, v, rot, other, torch.tensor([[0], [1]], dtype=I32, device=dev), lens, cu)
    assert torch.equal(got, want)
    lse = torch.zeros(5, 4, device=dev)
    for workspace in (None, fg.make_attention_workspace(dev)):
        out = fg.paged_attention(q, cache, table, lens, cu, lse=lse, workspace=workspace)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
