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


def test_more_rows_than_one_launch_holds(cuda_device):
    """A norm over heads of 128 columns of over 2^26 rows."""
    n, times, rest = 1 << 16, 1 << 10, 5
    g = synth.make_generator(3, cuda_device)
    X = torch.randn(n, 128, generator=g, device=cuda_device).to(BF16)
    w = torch.rand(128, generator=g, device=cuda_device) + 0.5
    Q, sa, _, rstd = fg.rmsnorm_quantize_1x128(X, w)
    many = torch.cat([X.repeat(times, 1), X[:rest]])
    q2, s2, _, r2 = fg.rmsnorm_quantize_1x128(many, w)
    assert bool((q2[: n * times].view(times, n, 128) == Q).all()) and torch.equal(q2[n * times:], Q[:rest])
    assert bool((s2[0, : n * times].view(times, n) == sa[0, :n]).all()) and torch.equal(s2[0, n * times: n * times + rest], sa[0, :rest])
    assert bool((r2[: n * times].view(times, n) == rstd).all()) and torch.equal(r2[n * times:], rstd[:rest])


def test_more_tokens_than_one_launch_holds(cuda_device):
    """Queries of over 2^25 tokens, two a workgroup: every 2^16 tokens are the same ones."""
    n, times, rest = 1 << 16, 1 << 9, 7
    T = n * times + rest
    g = synth.make_generator(4, cuda_device)
    q, k, v = (torch.randn(n, 1, 64, generator=g, device=cuda_device).to(BF16) for _ in range(3))
    rot = table_of(64, 32, cuda_device)
    positions = torch.randint(0, 64, (n,), generator=g, device=cuda_device, dtype=I32)

    def run(tokens, *inputs):
        pages = -(-tokens // 16)
        cache = fg.make_paged_kv_cache(pages, 1, 16, 64, device=cuda_device)
        table = torch.arange(pages, dtype=I32, device=cuda_device).view(1, pages)
        lens, cu = (torch.tensor(x, dtype=I32, device=cuda_device) for x in ([tokens], [0, tokens]))
        *rows, at = inputs
        return fg.rope_append_paged_kv(*rows, rot, cache, table, lens, cu, positions=at), cache

    def many(t):
        return torch.cat([t.repeat(times, *[1] * (t.dim() - 1)), t[:rest]])

    want, one = run(n, q, k, v, positions)
    got, all_ = run(T, many(q), many(k), many(v), many(positions))
    assert bool((got[: n * times].view(times, n, 64) == want.view(n, 64)).all()) and torch.equal(got[n * times:], want[:rest])
    pages = n // 16
    for a, b in zip(all_, one):
        assert bool((a[: pages * times].view(times, -1) == b.view(-1)).all())


def test_more_tiles_than_one_launch_holds(cuda_device):
    """Attention of 2^17 tokens of 2^10 heads in tiles of 16 rows, with as many places for tiles
    that hold the end of a sequence: every sequence is the same one."""
    B, n, H = 1 << 13, 16, 1 << 10
    g = synth.make_generator(5, cuda_device)
    cache = fg.make_paged_kv_cache(1, H, 16, 64, device=cuda_device)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 0x40, t.shape, generator=g, device=cuda_device, dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(0.25)
    q = torch.randn(n, H, 64, generator=g, device=cuda_device).to(BF16)

    def run(rows, b):
        return fg.paged_attention(rows, cache, torch.zeros(b, 1, dtype=I32, device=cuda_device),
                                  torch.full((b,), n, dtype=I32, device=cuda_device),
                                  torch.arange(b + 1, dtype=I32, device=cuda_device) * n)

    want = run(q, 1)
    assert (min(B, B * n) + B * n // 16) * H * 256 >= 1 << 32
    got = run(q.repeat(B, 1, 1), B).view(B, n, H, 64)
    assert all(bool((got[b: b + 1024] == want).all()) for b in range(0, B, 1024))
