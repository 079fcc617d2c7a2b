"""GPU parity of the norm and rotation of heads, and of its gradients, against the FP64 oracle.

Bounds, u = 2^-24: a head's sum of squares is a chain of 16 and four levels, so rstd is within 16 u
and a normed value within 24 u, 32 u of its magnitudes once turned (2^-19); a gradient is a product
of such values over such sums, 64 u of its magnitudes (2^-18); the weights' gradients add one term a
token and head. Outputs are rounded once."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from moe_grouped_gemm_fp32_amd import moe
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32
UNIT = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def fused(T, Hq, Hk, D, dtype, seed, dev, std=1.0):
    """Queries and keys as views of a projection's output."""
    g = synth.make_generator(seed, dev)
    x = (torch.randn(T, Hq + 2 * Hk, D, generator=g, device=dev) * std * torch.exp(torch.randn(D, generator=g, device=dev) * 0.3)).to(dtype)
    return x[:, :Hq], x[:, Hq:Hq + Hk]


def turns(n, rotated, dev):
    if rotated == 0:
        return None
    freq = 10000.0 ** (-torch.arange(rotated // 2, device=dev, dtype=torch.float64) * 2 / rotated)
    angle = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def weights_of(D, dtype, dev):
    g = synth.make_generator(77, dev)
    return [(1 + 0.3 * torch.randn(D, generator=g, device=dev)).to(dtype) for _ in range(2)]


def check(q, k, ws, table, at, eps=1e-6, interleaved=False, **kw):
    got = fg.qk_norm_rope(q, k, *ws, table, at, eps=eps, interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    for x, w, y in zip((q, k), ws, got):
        if x is None:
            assert y is None
            continue
        want, mag = mo.qk_norm_rope(f64(x), f64(w), f64(table), None if at is None else at.cpu().numpy(), eps, interleaved)
        assert y.dtype == x.dtype and y.shape == x.shape
        assert np.all(np.abs(f64(y) - want) <= UNIT[x.dtype] * np.abs(want) + 32 * U * mag)
    return got


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("T,Hq,Hk,D,rotated", [(1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (7, 8, 2, 256, 256), (65, 16, 4, 128, 64), (33, 3, 3, 64, 16),
                                               (9, 4, 2, 256, 48), (5, 7, 7, 64, 0), (300, 32, 8, 128, 128)])
def test_heads(cuda_device, dtype, wtype, T, Hq, Hk, D, rotated):
    q, k = fused(T, Hq, Hk, D, dtype, 1, cuda_device)
    ws, table = weights_of(D, wtype, cuda_device), turns(100, rotated, cuda_device)
    at = torch.randint(-5, 130, (T,), generator=synth.make_generator(2, cuda_device), device=cuda_device).to(I32)  # clamped to the table
    for interleaved in (False, True):
        want = check(q, k, ws, table, at, interleaved=interleaved)
        inplace = torch.cat([q, k], 1)
        got = fg.qk_norm_rope(inplace[:, :Hq], inplace[:, Hq:], *ws, table, at, interleaved=interleaved, q_out=inplace[:, :Hq],
                              k_out=inplace[:, Hq:])
        assert torch.equal(got[0], want[0]) and torch.equal(inplace[:, Hq:], want[1])
    check(q, None, [ws[0], None], table, None)
    got = check(None, k, [None, ws[1]], table, at, eps=1e-3)
    assert got[0] is None


def test_zero_rows_extremes_and_no_tokens(cuda_device):
    x = torch.zeros(4, 2, 64, device=cuda_device)
    x[1] = 1e-30
    x[2] = 1e17
    x[3, 0, 5] = 3e4
    ws, table = weights_of(64, FP32, cuda_device), turns(10, 64, cuda_device)
    check(x, x, ws, table, None)
    q, k = fg.qk_norm_rope(x[:0], x[:0], *ws, table)
    assert q.shape == k.shape == (0, 2, 64)
    none = fg.qk_norm_rope(x, x[:, :0], *ws, table)
    assert none[1].shape == (4, 0, 64)
    grad = fg.qk_norm_rope_backward(x, x[:, :0], x, x[:, :0], *ws, table)
    assert grad[1].shape == (4, 0, 64) and bool((grad[3] == 0).all())
    alone = fg.qk_norm_rope_backward(x, None, x, None, ws[0], None, table)
    assert torch.equal(grad[0], alone[0]) and torch.equal(grad[2], alone[2])


def test_the_append_of_what_comes_out(cuda_device):
    """Serving: normed and turned here, appended as they are; the same as the append's own rotation of
    normed heads."""
    T, Hq, Hk, D = 40, 4, 2, 128
    q, k = fused(T, Hq, Hk, D, BF16, 5, cuda_device)
    v = torch.randn(T, Hk, D, device=cuda_device).to(BF16)
    ws, table = weights_of(D, BF16, cuda_device), turns(64, D, cuda_device)
    bt = torch.arange(4, dtype=I32, device=cuda_device).view(1, 4)
    lens, cu = torch.tensor([50], dtype=I32, device=cuda_device), torch.tensor([0, T], dtype=I32, device=cuda_device)
    at = torch.arange(10, 50, dtype=I32, device=cuda_device)
    cache = fg.make_paged_kv_cache(4, Hk, 16, D)
    qo, ko = check(q, k, ws, table, at)
    assert fg.rope_append_paged_kv(None, ko, v, None, cache, bt, lens, cu) is None
    torch.cuda.synchronize()
    codes = cache.k.view(torch.float8_e4m3fn).float() * cache.k_scale[:, :, None, None]
    back = codes.transpose(1, 2).reshape(64, Hk, D)[10:50]
    assert bool(((back - ko.float()).abs() <= 2.0 ** -4 * ko.float().abs() + cache.k_scale.max() * 2.0 ** -10).all())


def check_grad(dq, dk, q, k, ws, table, at, interleaved=False, **kw):
    got = fg.qk_norm_rope_backward(dq, dk, q, k, *ws, table, at, interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    for dy, x, w, dx, dw in zip((dq, dk), (q, k), ws, got[:2], got[2:]):
        if dy is None:
            assert dx is None and dw is None
            continue
        want, ww, mag, magw = mo.qk_norm_rope_backward(f64(dy), f64(x), f64(w), f64(table), None if at is None else at.cpu().numpy(),
                                                       1e-6, interleaved)
        assert dx.dtype == x.dtype and dw.dtype == FP32
        assert np.all(np.abs(f64(dx) - want) <= UNIT[x.dtype] * np.abs(want) + 64 * U * mag)
        assert np.all(np.abs(f64(dw) - ww) <= (x.shape[0] * x.shape[1] + 64) * U * magw)
    return got


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("T,Hq,Hk,D,rotated", [(1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (7, 8, 2, 256, 256), (65, 16, 4, 128, 64), (33, 3, 3, 64, 16),
                                               (9, 4, 2, 256, 48), (5, 7, 7, 64, 0), (700, 32, 8, 128, 128)])
def test_gradients(cuda_device, dtype, wtype, T, Hq, Hk, D, rotated):
    q, k = fused(T, Hq, Hk, D, dtype, 1, cuda_device)
    dq, dk = (t.contiguous() for t in fused(T, Hq, Hk, D, dtype, 2, cuda_device, 0.1))
    ws, table = weights_of(D, wtype, cuda_device), turns(100, rotated, cuda_device)
    at = torch.randint(-5, 130, (T,), generator=synth.make_generator(3, cuda_device), device=cuda_device).to(I32)
    for interleaved in (False, True):
        got = check_grad(dq, dk, q, k, ws, table, at, interleaved)
        again = fg.qk_norm_rope_backward(dq, dk, q, k, *ws, table, at, interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    over, into = dq.clone(), torch.cat([q, k], 1)
    got2 = fg.qk_norm_rope_backward(over, dk, q, into[:, Hq:], *ws, table, at, interleaved=True, dq_out=over, dk_out=into[:, Hq:])
    assert torch.equal(got2[0], got[0]) and torch.equal(got2[1], got[1]) and torch.equal(into[:, :Hq], q)
    check_grad(dq, None, q, None, [ws[0], None], table, None)
    check_grad(None, dk, None, k, [None, ws[1]], table, at)


def test_gradients_against_differences(cuda_device):
    """Of the forward kernel in FP32, central differences of step 2^-5: off by roundings over the step
    (2^-19 of the loss's magnitude) and by the cubic term (step^2 times it)."""
    T, H, D, h = 2, 2, 64, 2.0 ** -5
    q, k = fused(T, H, H, D, FP32, 1, cuda_device)
    dq, dk = fused(T, H, H, D, FP32, 2, cuda_device)
    ws, table = weights_of(D, FP32, cuda_device), turns(8, 32, cuda_device)
    gq, gk, gqw, gkw = fg.qk_norm_rope_backward(dq, dk, q, k, *ws, table)

    def loss(q, k, ws):
        a, b = fg.qk_norm_rope(q, k, *ws, table)
        t = torch.cat([(a.double() * dq.double()).flatten(), (b.double() * dk.double()).flatten()])
        return float(t.sum()), float(t.abs().sum())

    mag = loss(q, k, ws)[1]
    for which, x, g in ((0, q, gq), (1, k, gk)):
        for i in ((0, 0, 0), (1, 1, 20), (0, 1, 63)):
            args = [[q.clone(), k.clone()] for _ in range(2)]
            args[0][which][i] += h
            args[1][which][i] -= h
            d = (loss(*args[0], ws)[0] - loss(*args[1], ws)[0]) / (2 * h)
            assert abs(d - float(g[i])) <= mag * (2.0 ** -19 / h + h * h)
    for which, g in ((0, gqw), (1, gkw)):
        for i in (0, 17, 50):
            up = [w.clone() for w in ws]
            up[which][i] += 1.0  # linear
            assert abs(loss(q, k, up)[0] - loss(q, k, ws)[0] - float(g[i])) <= mag * 2.0 ** -17


def test_gradients_of_no_tokens_and_workspace(cuda_device):
    x = torch.randn(30, 2, 64, device=cuda_device)
    ws = weights_of(64, FP32, cuda_device)
    got = fg.qk_norm_rope_backward(x[:0], x[:0], x[:0], x[:0], *ws)
    assert got[0].shape == (0, 2, 64) and bool((got[2] == 0).all()) and bool((got[3] == 0).all())
    need = moe._fn("fp8_qk_norm_rope_backward_workspace_size")(64)
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=cuda_device)
    a = fg.qk_norm_rope_backward(x, x, x, x, *ws, workspace=guard[:need])
    assert bool((guard[need:] == 0x5A).all())
    assert all(torch.equal(p, q) for p, q in zip(a, fg.qk_norm_rope_backward(x, x, x, x, *ws)))
    with pytest.raises(fg.Fp8GemmError):
        fg.qk_norm_rope_backward(x, x, x, x, *ws, workspace=guard[:16])


def test_refusals(cuda_device):
    q, k = fused(6, 4, 2, 64, BF16, 1, cuda_device)
    ws, table = weights_of(64, BF16, cuda_device), turns(8, 64, cuda_device)
    at = torch.zeros(6, dtype=I32, device=cuda_device)
    good = dict(q=q, k=k, q_weight=ws[0], k_weight=ws[1], cos_sin=table, positions=at)
    for bad in (dict(q=q.half()), dict(k=k.float()), dict(k=k[:5]), dict(q=q[:, ::2]), dict(q_weight=ws[0][:32]), dict(k_weight=ws[1].float()),
                dict(cos_sin=table.double()), dict(positions=at.long()), dict(positions=at[:5]), dict(q_out=k), dict(k=None, k_out=k)):
        with pytest.raises(ValueError):
            fg.qk_norm_rope(**{**good, **bad})
    for bad in (dict(q=q[..., :32].contiguous(), k=None, q_weight=ws[0][:32]), dict(cos_sin=turns(8, 24, cuda_device)), dict(eps=-1.0)):
        with pytest.raises(fg.Fp8GemmError):
            fg.qk_norm_rope(**{**good, **bad})
    with pytest.raises(TypeError):
        fg.qk_norm_rope(**{**good, "q_weight": None})
    for bad in (dict(dq=q[:5]), dict(dk=k.float()), dict(q=q[:, :2]), dict(dq=None, dq_out=q)):
        with pytest.raises(ValueError):
            fg.qk_norm_rope_backward(**{"dq": q, "dk": k, **good, **bad})
