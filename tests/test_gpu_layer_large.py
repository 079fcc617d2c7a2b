"""Calls whose rows do not fit the L2 caches are read as a stream, by instances of their own:
they give what the same rows give in smaller calls, bit for bit (the weight's gradient, whose
sums are grouped otherwise, within n 2^-24 of the terms' magnitudes, either side)."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("dtype,K,rows", [(BF16, 2048, 1509), (torch.float32, 1152, 1464), (BF16, 4992, 1060)])
def test_norm_and_gradient_of_many_rows(cuda_device, dtype, K, rows):
    size = 2 if dtype is BF16 else 4
    slices = 5
    M = slices * rows
    assert M * K * size * 2 > 32 << 20 and rows * K * size * 3 < 32 << 20 and rows > 1024
    g = synth.make_generator(1, cuda_device)
    x, r, dy, dh = (torch.randn(M, K, generator=g, device=cuda_device).to(dtype) for _ in range(4))
    w = torch.randn(K, generator=g, device=cuda_device).to(dtype)
    Q, sa, H, rstd = fg.rmsnorm_quantize_1x128(x, w, residual=r)
    dX, dW = fg.rmsnorm_backward(dy, H, rstd, w, dH=dh)
    total = torch.zeros(K, dtype=torch.float64, device=cuda_device)
    for i in range(slices):
        at = slice(i * rows, (i + 1) * rows)
        q1, s1, h1, r1 = fg.rmsnorm_quantize_1x128(x[at], w, residual=r[at])
        assert torch.equal(q1, Q[at]) and torch.equal(s1[:, :rows], sa[:, at]) and torch.equal(h1, H[at]) and torch.equal(r1, rstd[at])
        d1, w1 = fg.rmsnorm_backward(dy[at], h1, r1, w, dH=dh[at])
        assert torch.equal(d1, dX[at])
        total += w1.double()
    terms = (dy.double() * H.double() * rstd.double()[:, None]).abs().sum(dim=0)
    assert bool(((dW.double() - total).abs() <= 2 * M * 2.0 ** -24 * terms).all())


@pytest.mark.parametrize("D,P,interleaved", [(128, 64, False), (64, 16, True), (256, 128, False)])
def test_append_of_many_tokens(cuda_device, D, P, interleaved):
    Hq, Hkv = 2048 // D, 512 // D
    new = [2500, 1700, 2600]
    width = -(-max(new) // P)
    assert sum(new) * (Hq + 2 * Hkv) * D * 2 > 32 << 20 > max(new) * (Hq + 2 * Hkv) * D * 2
    g = synth.make_generator(2, cuda_device)
    T = sum(new)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=cuda_device).to(BF16)
    rot = torch.rand(max(new), D, generator=g, device=cuda_device) * 2 - 1
    table = torch.randperm(3 * width, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(3, width).to(cuda_device)
    lens = torch.tensor(new, dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0] + new, device=cuda_device).cumsum(0).to(torch.int32)

    def run(cache, rows, t, n, c):
        x = qkv[rows]
        return fg.rope_append_paged_kv(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], rot, cache, t, n, c, interleaved=interleaved)

    whole, parts = (fg.make_paged_kv_cache(3 * width, Hkv, P, D, device=cuda_device) for _ in range(2))
    q = run(whole, slice(0, T), table, lens, cu)
    for b in range(3):
        at = slice(sum(new[:b]), sum(new[:b + 1]))
        one = torch.tensor([0, new[b]], dtype=torch.int32, device=cuda_device)
        assert torch.equal(run(parts, at, table[b:b + 1], lens[b:b + 1], one), q[at])
    for a, b in zip(whole, parts):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K", [(1, 256), (37, 2048), (700, 1152), (1024, 4096)])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_gradient_of_few_rows_in_the_place_of_an_input(cuda_device, dtype, M, K):
    """dX may be dY or dH itself: the weight's gradient, summed beside it, is of dY as it was."""
    g = synth.make_generator(4, cuda_device)
    dy, h, dh = (torch.randn(M, K, generator=g, device=cuda_device).to(dtype) for _ in range(3))
    w = torch.randn(K, generator=g, device=cuda_device)
    _, _, _, rstd = fg.rmsnorm_quantize_1x128(h, w)
    dX, dW = fg.rmsnorm_backward(dy, h, rstd, w, dH=dh)
    terms = (dy.double() * h.double() * rstd.double()[:, None])
    bound = (M + 44) * 2.0 ** -24 * terms.abs().sum(dim=0)
    assert bool(((dW.double() - terms.sum(dim=0)).abs() <= bound).all())
    both = torch.cat([dy, dh], dim=1)  # views whose rows alternate, too
    for place in (dy.clone(), dh.clone(), both[:, :K], both[:, K:]):
        a = place if torch.equal(place, dy) else dy
        b = place if torch.equal(place, dh) else dh
        x, s = fg.rmsnorm_backward(a, h, rstd, w, dH=b, dX=place)
        assert torch.equal(x, dX)
        assert bool(((s.double() - terms.sum(dim=0)).abs() <= bound).all())
