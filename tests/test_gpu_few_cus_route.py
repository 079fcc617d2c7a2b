"""Routing on one compute unit, so that calls of some tens of rows take the kernels that the host
otherwise chooses for many thousands: the tests of test_gpu_moe_route.py, and others of more rows."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from oracle import moe_oracle as mo
from test_gpu_moe_route import *  # noqa: F401,F403  (its tests, its marker)
from test_gpu_moe_route import BF16, FP32, REL, check, f64, logits_of, pytestmark  # noqa: F401


@pytest.fixture(autouse=True)
def one_cu():
    fg.set_num_cus(1)
    yield
    fg.set_num_cus(0)


def check_decided(x, k, bias, scoring, groups, top_groups, best):
    """check(), but for rows in which 64 bits do not tell the last group kept from the first left
    out. Logits on a grid of u = 2^-24 and rounded biases give two groups the scores
    s(y) + s(y + 2u) and 2 s(y + u), which differ by u^2 s''(y) < 2^-51. A key below 2 in FP64
    is off by up to 2^-52 (exponential, sum, quotient and bias, of 2^-54 to 2^-53 each), a sum of
    two by 2^-51 and its own 2^-53, on either side: below 2^-49 the choice is open."""
    kw = dict(groups=groups, top_groups=top_groups, group_best=best)
    ids, w = fg.moe_route(x, k, bias=bias, scoring=scoring, **kw)
    again = fg.moe_route(x, k, bias=bias, scoring=scoring, scores=torch.empty_like(x), **kw)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)
    ri, rw, rs = mo.route(f64(x), k, f64(bias), scoring, **kw)
    decided = np.ones(len(ri), bool)
    if top_groups < groups:
        top = -np.sort(-(rs + f64(bias)).reshape(len(ri), groups, -1), axis=2)[:, :, :best]
        of = top.sum(2)
        order = np.argsort(-of, axis=1, kind="stable")[:, top_groups - 1:top_groups + 1]
        (kept, left), rows = order.T, np.arange(len(ri))
        near = (np.abs(of - of[rows, left][:, None]) <= 2.0 ** -49) & ~(top == top[rows, left][:, None]).all(2)
        decided = (of[rows, kept] - of[rows, left] > 2.0 ** -49) | ~near.any(1)
        assert decided.mean() > 0.5  # most rows are compared
    assert np.array_equal(ids.cpu().numpy()[decided], ri[decided])
    assert np.all(np.abs(f64(w) - rw)[decided] <= REL * np.abs(rw)[decided] + 2.0 ** -100)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", [(97, 33, 4, 1, 1, 1), (64, 64, 15, 1, 1, 1), (131, 64, 6, 8, 4, 2), (66, 64, 5, 16, 3, 2),
                                                          (101, 100, 8, 2, 1, 2), (99, 128, 8, 1, 1, 1), (120, 160, 6, 8, 3, 2),
                                                          (130, 256, 8, 8, 4, 2), (70, 256, 15, 1, 1, 1), (90, 240, 10, 15, 6, 1), (80, 256, 3, 16, 2, 2),
                                                          (75, 200, 12, 5, 2, 2), (65, 256, 16, 1, 1, 1)])
def test_more_rows(cuda_device, scoring, T, E, k, groups, top_groups, best):
    bias = torch.randn(E, generator=synth.make_generator(2, cuda_device), device=cuda_device) * 0.1
    for dtype in (FP32, BF16):
        x = logits_of(T, E, dtype, 13, cuda_device, pad=1)
        x[T // 2, E // 2:] = -float("inf")
        x[T // 3] = -float("inf")
        x[T // 3, 5:5 + k // 2] = 1.0  # fewer than k are left
        x[T - 1] = x[T - 1, 0]  # ties
        for b in (None, bias, torch.zeros_like(bias)):
            check(x, k, b, scoring, groups=groups, top_groups=top_groups, group_best=best, scale=-0.5)
    x = x.float()
    x[:, 1:] = x[:, :1] + torch.randint(-2, 3, (T, E - 1), generator=synth.make_generator(3, cuda_device), device=cuda_device) * 2.0 ** -24
    check(x, k, bias * 2.0 ** -18, scoring, groups=groups, top_groups=top_groups, group_best=best)
    check_decided(x, k, (bias * 2.0 ** -18).round(decimals=6), scoring, groups, top_groups, best)


@pytest.mark.parametrize("E", [64, 128, 256])
def test_pairs_that_differ_by_roundings(cuda_device, E):
    """Two near keys in each row, at the edge of the choice: decided among the candidates."""
    T, k = 128, 4
    g = synth.make_generator(5, cuda_device)
    x = torch.randn(T, E, generator=g, device=cuda_device)
    bias = torch.randn(E, generator=g, device=cuda_device) * 0.1
    key = torch.sigmoid(x.double()) + bias.double()
    order = key.argsort(dim=1, descending=True)
    rows = torch.arange(T, device=cuda_device)
    for a, b in ((k - 1, k), (0, 1)):
        want = key[rows, order[:, a]] - bias.double()[order[:, b]]  # the score that makes them equal
        fine = (want > 0.01) & (want < 0.99)
        x[rows[fine], order[fine, b]] = torch.logit(want[fine]).float()
    check(x, k, bias, "sigmoid")
    check(x, k, bias, "sigmoid", groups=4, top_groups=4)
