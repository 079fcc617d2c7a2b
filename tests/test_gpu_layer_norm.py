"""GPU parity of the residual RMS norm with 8-bit output, and of its gradients, against the
FP64 oracle.

Bounds, u = 2^-24 (FP32), K <= 65536. The sum of squares is a tree over at most 64 terms a
thread, 6 levels in a wave and 16 waves, so rstd is within 90 u relative, and y and s within
100 u < 2^-17. A code is the nearest to a quotient that is off by less than 2 * 2^-17
relative: half a step of the code's binade, plus that. Gradients: every term of dX is a
product of values off by less than 2^-17 relative, over sums of the same trees; dW adds M
terms in at most M + 40 roundings. Each output is rounded once (BF16: 2^-8 relative)."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import oracle
import synth
from moe_grouped_gemm_fp32_amd import layer
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
REL = 2.0 ** -17
UNIT = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
POS = oracle.E4M3_TABLE[:0x7F]  # increasing values of codes 0x00..0x7E


def half_step(a):
    hi = np.clip(np.searchsorted(POS, a, side="right"), 1, 0x7E)
    return 0.5 * (POS[hi] - POS[hi - 1])


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(M, K, dtype, seed, dev, pad=0, std=1.0):
    """[M, K] with a row stride of K + pad."""
    g = synth.make_generator(seed, dev)
    x = torch.randn(M, K, generator=g, device=dev) * std * torch.exp(torch.randn(K, generator=g, device=dev) * 0.5)
    out = torch.full((M, K + pad), float("nan"), dtype=dtype, device=dev)[:, :K]
    return out.copy_(x)


def check_norm(X, w, R, eps, got, Y=None):
    Q, sa, H, rstd = got
    torch.cuda.synchronize()
    M, K = X.shape
    h = X if R is None else (X.double() + R.double()).to(X.dtype)  # exact sums of two, rounded once
    if R is not None:
        assert torch.equal(H, h)
    y, r = lo.rmsnorm(f64(h), f64(w), eps)
    s = lo.block_scales(y)
    assert np.all(np.abs(f64(rstd) - r) <= REL * r)
    sg = f64(sa)[:, :M]
    assert np.all(np.abs(sg - s) <= REL * s)
    q = oracle.decode_e4m3(Q.cpu().numpy().view(np.uint8))
    want = y / np.repeat(s.T, 128, axis=1)
    assert np.all(np.abs(q - want) <= half_step(np.abs(want) * (1 + 2 * REL)) + 2 * REL * np.abs(want))
    if Y is not None:
        assert np.all(np.abs(f64(Y) - y) <= (UNIT[BF16] + REL) * np.abs(y))


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 384), (7, 1024), (3, 1152), (9, 2048), (2, 2176), (33, 7168), (1, 8192), (2, 8320),
                                 (3, 32768), (2, 32896), (1, 65536)])
def test_norm(cuda_device, dtype, wtype, M, K):
    X, R = rows(M, K, dtype, 1, cuda_device, 8), rows(M, K, dtype, 2, cuda_device, 16, 3.0)
    w = (1 + 0.2 * torch.randn(K, generator=synth.make_generator(3, cuda_device), device=cuda_device)).to(wtype)
    Y = torch.empty(M, K, dtype=BF16, device=cuda_device)
    check_norm(X, w, R, 1e-5, fg.rmsnorm_quantize_1x128(X, w, residual=R, eps=1e-5, Y=Y), Y)
    got = fg.rmsnorm_quantize_1x128(X, w)
    assert got[2] is X
    check_norm(X, w, None, 1e-6, got)


@pytest.mark.parametrize("M", [1, 2, 255, 1030])
def test_norm_rows_and_in_place_residual(cuda_device, M):
    """The residual stream updated in place, and an untouched scale padding."""
    K = 512
    X, R = rows(M, K, BF16, 4, cuda_device), rows(M, K, BF16, 5, cuda_device)
    w = torch.ones(K, device=cuda_device)
    want = fg.rmsnorm_quantize_1x128(X, w, residual=R)
    stream = R.clone()
    sa = torch.full((K // 128, fg.scale_ld(M) + 4), -7.0, device=cuda_device)
    got = fg.rmsnorm_quantize_1x128(X, w, residual=stream, H=stream, sa=sa)
    assert got[2] is stream and torch.equal(stream, want[2]) and torch.equal(got[0], want[0])
    assert torch.equal(sa[:, :M], want[1][:, :M]) and bool((sa[:, M:] == -7).all())
    other = X.clone()
    got = fg.rmsnorm_quantize_1x128(other, w, residual=R, H=other)
    assert torch.equal(other, want[2]) and torch.equal(got[0], want[0])


def test_norm_zero_rows_extremes_and_no_rows(cuda_device):
    K = 256
    X = torch.zeros(6, K, device=cuda_device)
    X[1] = 1e-30          # squares underflow: eps decides
    X[2, 5] = 3e4         # one large column
    X[3] = 1e18           # a large mean square
    X[4, :128] = 2.0      # a block of zeros beside one that is not
    w = torch.ones(K, device=cuda_device)
    w[7] = -4.0
    got = fg.rmsnorm_quantize_1x128(X, w)
    check_norm(X, w, None, 1e-6, got)
    assert bool(((got[0][0] & 0x7F) == 0).all()) and bool((got[1][:, 0] == 1).all()) and bool((got[1][1, 4] == 1).all())
    Q, sa, _, rstd = fg.rmsnorm_quantize_1x128(X[:0], w)
    assert Q.shape == (0, K) and rstd.numel() == 0


@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("M,K", [(1, 128), (6, 640), (9, 1536), (5, 2048), (700, 2176), (1100, 256), (3, 7168), (2, 16384), (3, 40960)])
def test_gradients(cuda_device, dtype, wtype, M, K):
    H, dY, dH = (rows(M, K, dtype, s, cuda_device, 8 * s) for s in (1, 2, 3))
    w = (1 + 0.2 * torch.randn(K, generator=synth.make_generator(3, cuda_device), device=cuda_device)).to(wtype)
    _, _, _, rstd = fg.rmsnorm_quantize_1x128(H, w)
    for extra in (dH, None):
        dX, dW = fg.rmsnorm_backward(dY, H, rstd, w, dH=extra)
        torch.cuda.synchronize()
        dx, dw, mag, magw = lo.rmsnorm_backward(f64(dY), f64(H), f64(rstd), f64(w), None if extra is None else f64(extra))
        assert dX.dtype == dtype and dW.dtype == FP32
        assert np.all(np.abs(f64(dX) - dx) <= UNIT[dtype] * np.abs(dx) + 2 * REL * mag)
        assert np.all(np.abs(f64(dW) - dw) <= (M + 44) * 2.0 ** -24 * magw)
        again = fg.rmsnorm_backward(dY, H, rstd, w, dH=extra)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dW)  # a fixed order
    inplace = dY.clone()
    got = fg.rmsnorm_backward(inplace, H, rstd, w, dH=dH, dX=inplace)
    assert torch.equal(got[0], fg.rmsnorm_backward(dY, H, rstd, w, dH=dH)[0])


def test_gradients_against_differences(cuda_device):
    """The forward kernel's own unquantised output, in central differences of step 1/8 (its
    values are rounded to BF16, so a smaller step would measure that). The loss weighs four
    outputs of a row: its error is two roundings of each over the step, and the cubic term
    of the difference, below step^2 times the outputs' magnitudes (rows of unit scale)."""
    M, K = 2, 128
    X = rows(M, K, FP32, 9, cuda_device)
    w = torch.linspace(0.5, 1.5, K, device=cuda_device)
    dY = torch.zeros(M, K, device=cuda_device)
    dY[:, [0, 1, 77, 127]] = torch.tensor([[1.0, -0.5, 0.7, 0.2], [0.3, 0.8, -1.0, 0.4]], device=cuda_device)

    def loss(x):
        Y = torch.empty(M, K, dtype=BF16, device=cuda_device)
        fg.rmsnorm_quantize_1x128(x, w, Y=Y)
        return (Y.double() * dY.double()).sum(dim=1), (Y.double().abs() * dY.double().abs()).sum(dim=1)

    _, _, _, rstd = fg.rmsnorm_quantize_1x128(X, w)
    dX, _ = fg.rmsnorm_backward(dY, X, rstd, w)
    step = 0.125
    for i, j in ((0, 0), (0, 77), (1, 1), (1, 77)):
        up, down = X.clone(), X.clone()
        up[i, j] += step
        down[i, j] -= step
        (a, mag), (b, _) = loss(up), loss(down)
        got, m = float(a[i] - b[i]) / (2 * step), float(mag[i])
        assert abs(got - float(dX[i, j])) <= 2.0 ** -8 * 2 * m / (2 * step) + step ** 2 * m
        assert abs(float(dX[i, j])) > 2 * (2.0 ** -8 * m / step + step ** 2 * m)  # the bound says something


def test_gradients_no_rows_and_workspace(cuda_device):
    K = 256
    w = torch.ones(K, device=cuda_device)
    e = torch.empty(0, K, device=cuda_device)
    dX, dW = fg.rmsnorm_backward(e, e, e[:, 0], w, dW=torch.full((K,), 3.0, device=cuda_device))
    assert dX.shape == (0, K) and bool((dW == 0).all())
    x = torch.randn(40, K, device=cuda_device)
    r = torch.ones(40, device=cuda_device)
    need = layer._fn("fp8_rmsnorm_backward_workspace_size")(40, K)
    with pytest.raises(fg.Fp8GemmError):
        fg.rmsnorm_backward(x, x, r, w, workspace=torch.empty(need - 16, dtype=torch.uint8, device=cuda_device))
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=cuda_device)
    fg.rmsnorm_backward(x, x, r, w, workspace=guard[:need])
    assert bool((guard[need:] == 0x5A).all())


def test_another_stream(cuda_device):
    X = rows(300, 1024, BF16, 11, cuda_device)
    w = torch.ones(1024, device=cuda_device)
    want = fg.rmsnorm_quantize_1x128(X, w)
    grad = fg.rmsnorm_backward(X, X, want[3], w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fg.rmsnorm_quantize_1x128(X, w, stream=s)
    grad2 = fg.rmsnorm_backward(X, X, got[3], w, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(grad2[0], grad[0]) and torch.equal(grad2[1], grad[1])
