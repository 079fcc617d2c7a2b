"""GPU parity of routing and of its gradient against the FP64 oracle. Choices are equal; weights
and scores are within bounds.

Bounds, u = 2^-24. A score's exponential is off by 4 u and by what the difference to the largest
logit was rounded by, |d| u with |d| <= 40 here; sums add at most 64 + 32 + 6 roundings, the rest a
few: below 200 u < 2^-16 relative (sigmoids: far less). What underflows is off by 2^-126.
Gradients: each term is a product of such values over such sums, twice that of its magnitude."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32
REL = 2.0 ** -16
UNIT = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def padded(t, pad, fill=float("nan")):
    """t with a row stride of its columns + pad."""
    out = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)[:, :t.shape[1]]
    return out.copy_(t)


def logits_of(T, E, dtype, seed, dev, pad=0, std=1.5):
    g = synth.make_generator(seed, dev)
    x = torch.randn(T, E, generator=g, device=dev) * std + torch.randn(E, generator=g, device=dev) * 0.5
    return padded(x.to(dtype), pad)


def check(x, k, bias=None, scoring="softmax", scores=True, **kw):
    T, E = x.shape
    s = torch.full((T, E + 3), -7.0, device=x.device)[:, :E] if scores else None
    ids, w = fg.moe_route(x, k, bias=bias, scoring=scoring, scores=s, **kw)
    torch.cuda.synchronize()
    ri, rw, rs = mo.route(f64(x), k, None if bias is None else f64(bias), scoring, **kw)
    assert ids.dtype == I32 and ids.shape == w.shape == (T, k)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.all(np.abs(f64(w) - rw) <= REL * np.abs(rw) + abs(kw.get("scale", 1.0)) * 2.0 ** -100)
    if scores:
        assert np.all(np.abs(f64(s) - rs) <= REL * rs + 2.0 ** -126)
        assert bool((s.as_strided((T, 3), (E + 3, 1), E) == -7).all())
        again = fg.moe_route(x, k, bias=bias, scoring=scoring, **kw)  # without them, the same
        assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    return ids, w


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (7, 8, 2), (65, 60, 6), (5, 64, 64), (33, 65, 4), (130, 256, 8), (4, 257, 9),
                                   (9, 1000, 16), (2, 1024, 64)])
def test_choice(cuda_device, dtype, scoring, T, E, k):
    x = logits_of(T, E, dtype, 1, cuda_device, pad=3)
    bias = torch.randn(E, generator=synth.make_generator(2, cuda_device), device=cuda_device) * 0.1
    for b in (None, bias, torch.zeros_like(bias)):
        check(x, k, b, scoring, scale=2.5)
        check(x, k, b, scoring, renormalize=False, scores=False)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (256, 8, 1, 8), (160, 8, 3, 6), (6, 3, 2, 3), (64, 64, 5, 5), (63, 21, 20, 7),
                                                   (1024, 2, 1, 10), (990, 33, 7, 20), (12, 4, 4, 4), (200, 5, 2, 30)])
def test_groups(cuda_device, best, scoring, E, groups, top_groups, k):
    bias = torch.randn(E, generator=synth.make_generator(2, cuda_device), device=cuda_device) * 0.1
    for dtype in (FP32, BF16):
        x = logits_of(41, E, dtype, 3, cuda_device)
        for b in (None, bias):
            check(x, k, b, scoring, groups=groups, top_groups=top_groups, group_best=best)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", [(203, 2, 1, 1, 1, 1), (1, 16, 16, 1, 1, 1), (17, 17, 3, 1, 1, 1), (98, 32, 4, 4, 2, 2),
                                                          (350, 48, 6, 3, 2, 2), (62, 64, 8, 8, 4, 2), (33, 64, 64, 1, 1, 1), (35, 64, 6, 16, 3, 1),
                                                          (500, 60, 7, 15, 4, 2), (31, 40, 40, 5, 5, 1), (64, 16, 2, 16, 9, 2),
                                                          (8201, 32, 5, 4, 2, 2), (8200, 20, 3, 2, 1, 1), (8300, 32, 15, 1, 1, 1)])
def test_few_experts(cuda_device, scoring, T, E, k, groups, top_groups, best):
    bias = torch.randn(E, generator=synth.make_generator(2, cuda_device), device=cuda_device) * 0.1
    for dtype in (FP32, BF16):
        x = logits_of(T, E, dtype, 13, cuda_device, pad=1)
        x[T // 2, E // 2:] = -float("inf")
        x[T - 1] = x[T - 1, 0]  # ties
        for b in (None, bias, torch.zeros_like(bias)):
            check(x, k, b, scoring, groups=groups, top_groups=top_groups, group_best=best, scale=-0.5)
    x = x.float()
    x[:, 1:] = x[:, :1] + torch.randint(-2, 3, (T, E - 1), generator=synth.make_generator(3, cuda_device), device=cuda_device) * 2.0 ** -24
    check(x, k, bias * 2.0 ** -18, scoring, groups=groups, top_groups=top_groups, group_best=best)


def test_many_rows_where_keys_lie_close(cuda_device):
    """Keys nearer to each other than FP32 can tell: spaced by 2^-30 of a score, and equal ones."""
    T, E, k = 400, 256, 8
    g = synth.make_generator(5, cuda_device)
    x = torch.randn(T, E, generator=g, device=cuda_device)
    bias = (0.5 - torch.sigmoid(x[0].double())).float()  # row 0: every key is 0.5 to the last bits
    x[1:] = x[0] + torch.randint(-2, 3, (T - 1, E), generator=g, device=cuda_device) * 2.0 ** -22
    check(x, k, bias, "sigmoid")
    check(x, k, bias, "sigmoid", groups=8, top_groups=3, group_best=2)
    x = torch.randint(0, 3, (T, E), generator=g, device=cuda_device).float()  # ties everywhere
    for scoring in ("softmax", "sigmoid"):
        check(x, k, None, scoring)
        check(x, k, torch.full((E,), 0.25, device=cuda_device), scoring, groups=16, top_groups=5, group_best=2)
    y = torch.full((3, E), 37.0, device=cuda_device)  # sigmoids that round to 1
    y[1, 99], y[2, 200] = 38.0, 37.000004
    assert fg.moe_route(y, 1, scoring="sigmoid")[0].flatten().tolist() == [0, 99, 200]


@pytest.mark.parametrize("center", [-60.0, -30.0, -12.0, 0.0, 9.0])
def test_keys_that_differ_by_a_few_roundings_at_every_size(cuda_device, center):
    """Sigmoids of any magnitude, made almost equal by their biases."""
    T, E, k = 300, 128, 8
    g = synth.make_generator(11, cuda_device)
    x = center + torch.randn(T, E, generator=g, device=cuda_device) * 1e-3
    base = torch.sigmoid(x[0].double())
    bias = (base.max() * 2 - base).float()
    x[1:] = x[0] + torch.randint(-3, 4, (T - 1, E), generator=g, device=cuda_device) * abs(center) * 2.0 ** -23
    check(x, k, bias, "sigmoid")
    check(x, k, bias, "sigmoid", groups=4, top_groups=2, group_best=2)
    check(x, k, bias, "softmax")


@pytest.mark.parametrize("E", [16, 32, 64, 128, 256, 300])
@pytest.mark.parametrize("k", [1, 3, 10])
def test_a_larger_key_behind_equal_ones(cuda_device, E, k):
    """Many equal keys, and one that is larger by less than a rounding of theirs, after all of them."""
    T = 70
    x = torch.zeros(T, E, device=cuda_device)
    bias = torch.full((E,), 0.1, device=cuda_device)
    bias[E - 1] = torch.nextafter(bias[0], torch.tensor(1.0, device=cuda_device))
    ids, _ = check(x, k, bias, "sigmoid")
    assert ids[0].tolist() == [E - 1, *range(k - 1)]
    bias[E // 2:] = -float("inf")  # as few equal ones as may be candidates
    bias[E // 2 - 1] = torch.nextafter(bias[0], torch.tensor(1.0, device=cuda_device))
    check(x, min(k, E // 2), bias, "sigmoid")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(16, 1), (32, 4), (64, 1), (128, 8), (256, 1), (256, 8), (300, 3)])
def test_biases_without_bounds(cuda_device, E, groups, scoring):
    """Keys of +inf are equal, those of -inf are never chosen, those of FP32's largest are above others."""
    T, k = 70, 4
    x = logits_of(T, E, FP32, 21, cuda_device)
    kw = dict(groups=groups, top_groups=max(groups // 2, 1), group_best=2 if groups > 1 else 1)
    for value in (float("inf"), torch.finfo(FP32).max, -torch.finfo(FP32).max):
        for some in (slice(1, None, 3), slice(0, E), slice(E // 2 - 1, E // 2 + 1)):
            bias = torch.zeros(E, device=cuda_device)
            bias[some] = value
            bias[2] = -float("inf")
            check(x, k, bias, scoring, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_experts_that_are_not_there(cuda_device, scoring):
    T, E, k = 50, 96, 6
    x = logits_of(T, E, FP32, 6, cuda_device)
    x[:, ::3] = -float("inf")
    x[7] = -float("inf")
    x[8, 3:] = -float("inf")  # two are left
    x[9, :48] = -float("inf")
    bias = torch.zeros(E, device=cuda_device)
    bias[1] = -float("inf")
    for b in (None, bias):
        check(x, k, b, scoring)
        check(x, k, b, scoring, groups=4, top_groups=2, group_best=2)
    ids, w = fg.moe_route(x, k, scoring=scoring)
    assert ids[7].tolist() == [-1] * k and w[7].tolist() == [0.0] * k and ids[8].tolist()[2:] == [-1] * (k - 2)
    low = torch.full((2, E), torch.finfo(FP32).min, device=cuda_device)  # a mask of the type's lowest value is a number
    low[1, 5] = 0.0
    ids, w = fg.moe_route(low, 2, scoring="softmax")
    assert ids.tolist() == [[0, 1], [5, 0]] and w.tolist() == [[0.5, 0.5], [1.0, 0.0]]


def test_extreme_logits(cuda_device):
    x = torch.tensor([[300.0, -300.0, 0.0, 88.0], [1e30, 1e30, -1e30, 0.0], [-1e4, -2e4, -1e4, -3e4]], device=cuda_device)
    for scoring in ("softmax", "sigmoid"):
        ids, w = fg.moe_route(x, 2, scoring=scoring, renormalize=False)
        ri, rw, _ = mo.route(f64(x), 2, None, scoring, renormalize=False)
        assert np.array_equal(ids.cpu().numpy(), ri) and np.allclose(f64(w), rw, rtol=REL, atol=2.0 ** -126)
    x[0, 1], x[1, 3] = float("nan"), float("inf")  # the numbers of experts stay numbers of experts
    ids, w = fg.moe_route(x, 4, bias=torch.zeros(4, device=cuda_device), scoring="softmax")
    assert sorted(ids[0].tolist()) == [0, 1, 2, 3] and bool(torch.isnan(w[:2]).all())
    ids, w = fg.moe_route(x, 4, scoring="sigmoid")
    assert ids[0].tolist() == [0, 3, 2, 1] and bool(torch.isnan(w[0]).all()) and ids[1, 0] == 3


def test_no_rows_outputs_given_and_refusals(cuda_device):
    x = logits_of(6, 16, FP32, 1, cuda_device)
    ids, w = fg.moe_route(x[:0], 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    ids, w = torch.empty(6, 3, dtype=I32, device=cuda_device), torch.empty(6, 3, device=cuda_device)
    got = fg.moe_route(x, 3, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    for bad in (dict(top_k=0), dict(top_k=17), dict(scoring="relu"), dict(bias=w[0]), dict(ids=w), dict(weights=w[:, :2]),
                dict(scores=x[:, :8]), dict(ids=ids[:, ::2])):
        with pytest.raises(ValueError):
            fg.moe_route(x, **{"top_k": 3, **bad})
    for bad in (dict(groups=3), dict(groups=4, top_groups=5), dict(group_best=3), dict(scale=float("nan"))):
        with pytest.raises(fg.Fp8GemmError):
            fg.moe_route(x, 3, **bad)
    with pytest.raises(ValueError):
        fg.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        fg.moe_route(x.t(), 2)


def check_grad(dw, x, ids, scoring, renormalize, scale, ds, **kw):
    dx = fg.moe_route_backward(dw, x, ids, scoring=scoring, renormalize=renormalize, scale=scale, dscores=ds, **kw)
    torch.cuda.synchronize()
    want, mag = mo.route_backward(f64(dw), f64(x), ids.cpu().numpy(), scoring, renormalize, scale, f64(ds))
    assert dx.dtype == x.dtype
    assert np.all(np.abs(f64(dx) - want) <= UNIT[x.dtype] * np.abs(want) + 2 * REL * mag + 2.0 ** -126)
    return dx


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (70, 60, 6), (5, 64, 64), (130, 256, 8), (4, 257, 9), (3, 1024, 64), (33, 16, 16),
                                   (31, 32, 17), (18, 33, 4), (1000, 64, 8)])
def test_gradient(cuda_device, dtype, scoring, T, E, k):
    x = logits_of(T, E, dtype, 1, cuda_device, pad=5)
    g = synth.make_generator(3, cuda_device)
    dw, ds = torch.randn(T, k, generator=g, device=cuda_device), padded(torch.randn(T, E, generator=g, device=cuda_device) * 0.1, 2)
    for renormalize in (True, False):
        ids, _ = fg.moe_route(x, k, scoring=scoring, renormalize=renormalize, scale=2.5)
        for extra in (ds, None):
            dx = check_grad(dw, x, ids, scoring, renormalize, 2.5, extra)
            assert torch.equal(dx, fg.moe_route_backward(dw, x, ids, scoring, renormalize, 2.5, extra))
    inplace = x.clone()
    got = fg.moe_route_backward(dw, inplace, ids, scoring, False, 2.5, dlogits=inplace)
    assert got is inplace and torch.equal(got, dx)


def test_gradient_of_choices_that_are_none_or_named_twice(cuda_device):
    x = logits_of(4, 12, FP32, 8, cuda_device)
    x[3] = -float("inf")
    x[2, 6:] = -float("inf")
    ids = torch.tensor([[3, -1, 5], [-1, -1, -1], [2, 2, 99], [-1, -1, -1]], dtype=I32, device=cuda_device)
    dw = torch.randn(4, 3, device=cuda_device)
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            dx = check_grad(dw, x, ids, scoring, renormalize, 1.5, None)
            assert bool((dx[[1, 3]] == 0).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_against_differences(cuda_device, scoring):
    """Of the forward kernel, in central differences of step 2^-6: the weights (below 1, FP32) are off
    by 2^-16, and the cubic term is below step^2 times the weights' third derivative (below 8)."""
    T, E, k, h = 2, 10, 4, 2.0 ** -6
    x = logits_of(T, E, FP32, 9, cuda_device, std=1.0)
    ids, _ = fg.moe_route(x, k, scoring=scoring)
    dw = torch.tensor([[1.0, -0.5, 0.25, 2.0]] * T, device=cuda_device)
    dx = f64(fg.moe_route_backward(dw, x, ids, scoring=scoring))
    for t in range(T):
        for e in ids[t].tolist():
            got = 0.0
            for sign in (1, -1):
                y = x.clone()
                y[t, e] += sign * h
                i2, w2 = fg.moe_route(y, k, scoring=scoring)
                by_id = dict(zip(i2[t].tolist(), f64(w2)[t]))
                if set(by_id) != set(ids[t].tolist()):
                    break  # the step changes the choice
                got += sign * sum(float(dw[t, j]) * by_id[i] for j, i in enumerate(ids[t].tolist()))
            else:
                assert abs(got / (2 * h) - dx[t, e]) <= 3.75 * (REL / h + 8 * h * h)


def test_gradient_refusals(cuda_device):
    x = logits_of(6, 16, FP32, 1, cuda_device)
    ids, w = fg.moe_route(x, 3)
    assert fg.moe_route_backward(w[:0], x[:0], ids[:0]).shape == (0, 16)
    for bad in (dict(dweights=w[:, :2]), dict(ids=w), dict(dscores=w), dict(dlogits=x.bfloat16()), dict(scoring="top")):
        with pytest.raises(ValueError):
            fg.moe_route_backward(**{"dweights": w, "logits": x, "ids": ids, **bad})
