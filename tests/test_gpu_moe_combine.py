"""GPU parity of the combination of experts' rows, and of its gradients, against the FP64 oracle.

Bounds, u = 2^-24: a sum of top_k products is off by (top_k + 2) u of the terms' magnitudes, a dot
product over N columns by (N / 64 + 16) u (a lane's chain, six levels, four waves), each output by
half a step of its type."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32
UNIT = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rows_of(M, N, dtype, seed, dev, pad=0):
    g = synth.make_generator(seed, dev)
    return torch.full((M, N + pad), float("nan"), dtype=dtype, device=dev)[:, :N].copy_(torch.randn(M, N, generator=g, device=dev))


def places(T, k, rows, seed, dev, none=0.2):
    """Distinct rows for the choices, some without one."""
    g = synth.make_generator(seed, dev)
    at = torch.full((T * k,), -1, dtype=I32, device=dev)
    n = min(rows, T * k)
    at[torch.randperm(T * k, generator=g, device=dev)[:n]] = torch.randperm(rows, generator=g, device=dev)[:n].to(I32)
    at[torch.rand(T * k, generator=g, device=dev) < none] = -1
    return at.view(T, k)


def check(Y, at, w=None, C=None, **kw):
    out = fg.moe_combine(Y, at, w, C=C, **kw)
    torch.cuda.synchronize()
    N = Y.shape[-1]
    want, mag = mo.combine(f64(Y).reshape(-1, N), at.cpu().numpy(), f64(w), f64(C))
    assert out.dtype == Y.dtype and out.shape == (at.shape[0], N)
    assert np.all(np.abs(f64(out) - want) <= UNIT[Y.dtype] * np.abs(want) + (at.shape[1] + 2) * U * mag)
    return out


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,k,rows,N", [(1, 1, 1, 8), (1, 8, 1024, 7168), (3, 2, 128, 504), (5, 9, 100, 520), (64, 8, 600, 2048), (7, 64, 640, 136),
                                        (130, 3, 512, 1032), (40, 6, 333, 256)])
def test_combine(cuda_device, dtype, T, k, rows, N):
    Y, C = rows_of(rows, N, dtype, 1, cuda_device, 8), rows_of(T, N, dtype, 2, cuda_device, 16)
    at = places(T, k, rows, 3, cuda_device)
    w = torch.randn(T, k, generator=synth.make_generator(4, cuda_device), device=cuda_device)
    want = check(Y, at, w, C)
    check(Y, at, w)
    check(Y, at)  # the gradient of a dispatch
    stream = C.clone()
    assert fg.moe_combine(Y, at, w, C=stream, out=stream) is stream and torch.equal(stream, want)


def test_a_row_twice_none_and_nonsense(cuda_device):
    Y = rows_of(10, 64, FP32, 1, cuda_device)
    at = torch.tensor([[3, 3, 3], [-1, -1, -1], [10, 1 << 30, -(1 << 31)], [9, -5, 0]], dtype=I32, device=cuda_device)
    w = torch.randn(4, 3, device=cuda_device)
    out = check(Y, at, w)
    assert bool((out[1:3] == 0).all())
    Y[5] = float("nan")  # rows that nobody names, and weights without a row, may hold anything
    w[1:3] = float("nan")
    assert torch.equal(check(Y, at, torch.nan_to_num(w)), fg.moe_combine(Y, at, w))
    assert bool((fg.moe_combine(Y[:0], at, w) == 0).all())
    assert fg.moe_combine(Y, at[:0], w[:0]).shape == (0, 64)


def test_masked_rows_and_strides(cuda_device):
    E, max_m, N = 6, 5, 96
    base = rows_of(E * max_m, N + 24, BF16, 2, cuda_device)
    Y = base.view(E, max_m, N + 24)[..., :N]
    at = places(11, 3, E * max_m, 5, cuda_device)
    w = torch.rand(11, 3, device=cuda_device)
    out = check(Y, at, w)
    assert torch.equal(out, fg.moe_combine(Y.reshape(-1, N), at, w))


def check_grad(dO, Y, at, w, dY=None):
    before = None if dY is None else dY.clone()
    y64 = f64(Y).reshape(-1, Y.shape[-1])
    gy, dw = fg.moe_combine_backward(dO, Y, at, w, dY=dY)
    torch.cuda.synchronize()
    N = dO.shape[1]
    rows, want, mag = mo.combine_backward(f64(dO), y64, at.cpu().numpy(), f64(w))
    assert dw.dtype == FP32 and np.all(np.abs(f64(dw) - want) <= (N / 64 + 16) * U * mag)
    flat = f64(gy).reshape(-1, N)
    for p, row in rows.items():
        assert np.all(np.abs(flat[p] - row) <= (UNIT[Y.dtype] + U) * np.abs(row))
    if before is not None:
        rest = [p for p in range(len(flat)) if p not in rows]
        assert np.array_equal(flat[rest], f64(before).reshape(-1, N)[rest], equal_nan=True)
    return gy, dw


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,k,rows,N", [(1, 1, 1, 8), (1, 8, 1024, 7168), (3, 2, 128, 504), (5, 9, 100, 520), (64, 8, 600, 2048), (7, 64, 640, 136),
                                        (130, 3, 512, 1032), (40, 17, 333, 256)])
def test_gradients(cuda_device, dtype, T, k, rows, N):
    Y, dO = rows_of(rows, N, dtype, 1, cuda_device, 8), rows_of(T, N, dtype, 2, cuda_device, 16)
    at = places(T, k, rows, 3, cuda_device)
    w = torch.randn(T, k, generator=synth.make_generator(4, cuda_device), device=cuda_device)
    dY = torch.full((rows, N + 8), 5.0, dtype=dtype, device=cuda_device)[:, :N]
    gy, dw = check_grad(dO, Y, at, w, dY)
    assert gy is dY and torch.equal(dw, fg.moe_combine_backward(dO, Y, at, w)[1])
    none, alone = fg.moe_combine_backward(dO, Y, at, w, rows=False)
    assert none is None and torch.equal(alone, dw)
    inplace = Y.clone()
    gy2, dw2 = check_grad(dO, inplace, at, w, inplace)
    named = at[at >= 0].long()
    assert torch.equal(gy2[named], gy[named]) and torch.equal(dw2, dw)


def test_gradients_of_no_rows_and_masked_rows(cuda_device):
    E, max_m, N = 6, 5, 96
    Y, dO = rows_of(E * max_m, N, FP32, 2, cuda_device).view(E, max_m, N), rows_of(11, N, FP32, 3, cuda_device)
    at = places(11, 3, E * max_m, 5, cuda_device)
    w = torch.rand(11, 3, device=cuda_device)
    gy, _ = check_grad(dO, Y, at, w, torch.zeros_like(Y))
    assert gy.shape == Y.shape
    none = torch.full_like(at, -1)
    gy, dw = fg.moe_combine_backward(dO, Y, none, w, dY=torch.ones_like(Y))
    assert bool((gy == 1).all()) and bool((dw == 0).all())
    gy, dw = fg.moe_combine_backward(dO[:0], Y, at[:0], w[:0])
    assert dw.shape == (0, 3)
    # of the dispatch: what a token's rows give, summed
    back = fg.moe_combine(gy.zero_().add_(1.0), at)
    assert torch.equal(back, (at >= 0).sum(1, keepdim=True).float().expand(-1, N))


def test_gradients_against_differences(cuda_device):
    """Linear in each argument: a difference of any step is exact but for roundings (FP32, values
    below 8, sums of 2 x 24 terms: 2^-16)."""
    Y, dO = rows_of(7, 24, FP32, 1, cuda_device), rows_of(4, 24, FP32, 2, cuda_device)
    at = places(4, 2, 7, 3, cuda_device, none=0.0)
    w = torch.rand(4, 2, device=cuda_device)
    gy, dw = fg.moe_combine_backward(dO, Y, at, w, dY=torch.zeros_like(Y))

    def loss(Y, w):
        return float((fg.moe_combine(Y, at, w).double() * dO.double()).sum())

    for i, j in ((0, 0), (3, 23), (6, 11)):
        up = Y.clone()
        up[i, j] += 1.0
        assert abs(loss(up, w) - loss(Y, w) - float(gy[i, j])) < 2.0 ** -12
    for i, j in ((0, 0), (3, 1)):
        up = w.clone()
        up[i, j] += 1.0
        assert abs(loss(Y, up) - loss(Y, w) - float(dw[i, j])) < 2.0 ** -12


def test_refusals(cuda_device):
    Y, dO = rows_of(16, 64, BF16, 1, cuda_device), rows_of(4, 64, BF16, 2, cuda_device)
    at = places(4, 2, 16, 3, cuda_device)
    w = torch.rand(4, 2, device=cuda_device)
    for bad in (dict(Y=Y.half()), dict(Y=Y.t()), dict(positions=at.long()), dict(positions=at[0]), dict(weights=w[:3]), dict(weights=w.double()),
                dict(C=dO.float()), dict(C=dO[:3]), dict(out=dO[:, :32]), dict(out=dO.float())):
        with pytest.raises(ValueError):
            fg.moe_combine(**{"Y": Y, "positions": at, "weights": w, **bad})
    with pytest.raises(fg.Fp8GemmError):
        fg.moe_combine(Y[:, :12].contiguous(), at, w)
    for bad in (dict(dO=dO.float()), dict(dO=dO[:3]), dict(Y=Y[:, :32]), dict(weights=w[:3]), dict(dY=Y[:3]), dict(dY=Y.float()),
                dict(dweights=w[:3]), dict(dY=Y, rows=False)):
        with pytest.raises(ValueError):
            fg.moe_combine_backward(**{"dO": dO, "Y": Y, "positions": at, "weights": w, **bad})
