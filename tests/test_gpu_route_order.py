"""The order that routing goes by where FP32 leaves it open, of one row a wave and of four: group
scores whose keys cancel or pass FP32's numbers, logits whose scores are the same, NaN,
scores below the normal numbers.

A decision is compared where 64 bits tell it: scores are off by less than 2^-50, keys and their
sums by 2^-53 of the keys' magnitudes, on the kernel's side and on the oracle's, so that scores
of groups 2^-48 (1 + the largest bias) apart are told."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import synth
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

FP32 = torch.float32


@pytest.fixture(params=[0, 1], ids=["all CUs", "one CU"])
def cus(request):
    """On one compute unit the host takes four rows a wave for 64 rows and more."""
    fg.set_num_cus(request.param)
    yield request.param
    fg.set_num_cus(0)


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("size", [0.5, 1.0, 5.0, 100.0])
@pytest.mark.parametrize("scoring,center", [("sigmoid", -4.0), ("sigmoid", -8.0), ("softmax", 0.0)])
@pytest.mark.parametrize("E,groups,top_groups", [(4, 2, 1), (16, 8, 3), (64, 2, 1), (64, 8, 3), (256, 8, 4), (512, 4, 2)])
def test_groups_whose_two_keys_cancel(cuda_device, cus, E, groups, top_groups, scoring, center, size):
    """In each group one bias of +size and one of -size, and scores whose sums are nearly the same."""
    T = 300
    g = synth.make_generator(7, cuda_device)
    x = center + 0.3 * torch.randn(T, groups, E // groups, generator=g, device=cuda_device, dtype=torch.float64).clamp(-2, 2)
    bias = torch.full((groups, E // groups), -4 * size, device=cuda_device)
    bias[:, 0], bias[:, -1] = size, -size
    if scoring == "sigmoid":
        total = 2.2 * torch.sigmoid(torch.tensor(center, dtype=torch.float64))
        x[..., -1] = torch.logit(total - torch.sigmoid(x[..., 0].float().double()))
    else:
        x[..., -1] = torch.log(2.2 - x[..., 0].float().double().exp())
    x, bias = x.view(T, E).float(), bias.view(E)
    ids, w = fg.moe_route(x, 2, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups, group_best=2)
    ri, rw, rs = mo.route(f64(x), 2, f64(bias), scoring, groups=groups, top_groups=top_groups, group_best=2)
    keys = -np.sort(-(rs + f64(bias)).reshape(T, groups, -1), axis=2)
    of = -np.sort(-keys[:, :, :2].sum(2), axis=1)
    decided = of[:, top_groups - 1] - of[:, top_groups] > 2.0 ** -48 * (1 + size)
    assert decided.mean() > 0.9
    assert np.array_equal(ids.cpu().numpy()[decided], ri[decided])
    assert np.all(np.abs(f64(w) - rw)[decided] <= 2.0 ** -16 * rw[decided])


def test_one_row_whose_group_scores_cancel(cuda_device):
    """Scores 8.05306e-4 and 8.05238e-4: the first group. Keys near 1 and -1 are rounded by 6e-8."""
    x = torch.tensor([[-7.774, -7.862, -8.271, -7.506]], device=cuda_device)
    bias = torch.tensor([1.0, -1.0, 1.0, -1.0], device=cuda_device)
    ids, _ = fg.moe_route(x, 2, bias=bias, scoring="sigmoid", groups=2, top_groups=1, group_best=2)
    assert ids.tolist() == [[0, 1]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(4, 2), (16, 4), (32, 4), (64, 2), (64, 8), (256, 8), (512, 4)])
def test_group_scores_that_pass_fp32(cuda_device, cus, E, groups, scoring):
    """Sums of two keys below FP32's lowest value or above its largest: a group without experts is no
    better than those, and their order is that of the sums."""
    T, size, big = 70, E // groups, torch.finfo(FP32).max
    x = torch.randn(T, E, generator=synth.make_generator(3, cuda_device), device=cuda_device)
    kw = dict(groups=groups, group_best=2)
    for top_groups in (1, max(1, groups // 2)):
        for sign in (-1.0, 1.0):
            for parts in ((1.0, 1.0), (1.0, 0.9), (0.9, 1.0), (1.0, 0.4)):
                bias = torch.zeros(groups, size, device=cuda_device)
                for i in range(groups):
                    bias[i] = sign * big * parts[i % 2]
                for empty in (False, True):
                    y = x.clone()
                    if empty:
                        y[:, :size] = -float("inf")
                    ids, w = fg.moe_route(y, 2, bias=bias.view(E), scoring=scoring, top_groups=top_groups, **kw)
                    ri, rw, _ = mo.route(f64(y), 2, f64(bias.view(E)), scoring, top_groups=top_groups, **kw)
                    assert np.array_equal(ids.cpu().numpy(), ri), (top_groups, sign, parts, empty)
                    assert np.all(np.abs(f64(w) - rw) <= 2.0 ** -16 * rw + 2.0 ** -100)


@pytest.mark.parametrize("scoring,low", [("sigmoid", 37.5), ("softmax", -900.0)])
@pytest.mark.parametrize("E,groups,top_groups", [(4, 2, 1), (32, 4, 2), (64, 2, 1), (64, 16, 7), (256, 8, 4), (512, 4, 2)])
def test_experts_without_a_bias_go_by_their_logits(cuda_device, cus, E, groups, top_groups, scoring, low):
    """Scores of 1 and of 0 to the last bit, whose logits differ, in groups that take two keys."""
    T, size = 90, E // groups
    x = low + torch.rand(T, E, generator=synth.make_generator(4, cuda_device), device=cuda_device) * 8
    if scoring == "softmax":
        x[:, ::size] = 0.0  # one expert of each group has the scores
    k = min(6, top_groups * size)
    ids, w = fg.moe_route(x, k, scoring=scoring, groups=groups, top_groups=top_groups, group_best=2)
    ri, rw, _ = mo.route(f64(x), k, None, scoring, groups=groups, top_groups=top_groups, group_best=2)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.all(np.abs(f64(w) - rw) <= 2.0 ** -16 * rw)


@pytest.mark.parametrize("E", [3, 16, 32, 64, 256, 300])
def test_nan_comes_after_every_number(cuda_device, cus, E):
    """Also after FP32's lowest, which a mask may use; and before what is never chosen."""
    T, lowest, nan, none = 70, torch.finfo(FP32).min, float("nan"), -float("inf")
    x = torch.full((T, E), none, device=cuda_device)
    x[:, 0], x[:, 1], x[:, E - 1] = nan, lowest, 1.0
    for scoring in ("sigmoid", "softmax"):
        assert fg.moe_route(x, 3, scoring=scoring)[0].tolist() == [[E - 1, 1, 0]] * T
    assert fg.moe_route(x, 2, scoring="sigmoid")[1].isnan().sum() == 0
    y = torch.where(x == lowest, -2e30, x)
    assert fg.moe_route(y, 3, scoring="sigmoid")[0].tolist() == [[E - 1, 1, 0]] * T
    x[:, 1] = 0.0
    for value in (lowest, -2e30):
        bias = torch.zeros(E, device=cuda_device)
        bias[1] = value
        assert fg.moe_route(x, 3, bias=bias, scoring="sigmoid")[0].tolist() == [[E - 1, 1, 0]] * T
        bias[1], bias[0] = nan, value
        z = torch.where(x.isnan(), 0.0, x)  # a bias that is none
        assert fg.moe_route(z, 3, bias=bias, scoring="sigmoid")[0].tolist() == [[E - 1, 0, 1]] * T


@pytest.mark.parametrize("E,groups", [(4, 2), (16, 4), (64, 2), (256, 8), (512, 4)])
def test_groups_of_nan_come_last(cuda_device, cus, E, groups):
    T, size, lowest = 70, E // groups, torch.finfo(FP32).min
    x = torch.zeros(T, groups, size, device=cuda_device)
    x[:, :-1] = float("nan")
    for bias in (None, torch.zeros(E, device=cuda_device), torch.full((E,), lowest, device=cuda_device)):
        for best in (1, 2):
            ids, _ = fg.moe_route(x.view(T, E), 2, bias=bias, scoring="sigmoid", groups=groups, top_groups=1, group_best=best)
            assert ids.tolist() == [[E - size, E - size + 1]] * T
    x[:, -1] = lowest
    ids, _ = fg.moe_route(x.view(T, E), 2, scoring="sigmoid", groups=groups, top_groups=1)
    assert ids.tolist() == [[E - size, E - size + 1]] * T


@pytest.mark.parametrize("E", [16, 32, 64, 256, 300])
def test_scores_below_the_normal_numbers(cuda_device, cus, E):
    """sigmoid(-87.5) = 1e-38 is nothing to the card, and larger than a bias of 2e-39."""
    T = 70
    x = torch.full((T, E), -100.0, device=cuda_device)
    x[:, E - 1] = -87.5
    bias = torch.zeros(E, device=cuda_device)
    bias[:E // 2] = 2e-39
    ids, _ = fg.moe_route(x, 3, bias=bias, scoring="sigmoid")
    assert ids.tolist() == [[E - 1, 0, 1]] * T


@pytest.mark.parametrize("E", [4, 64, 256])
@pytest.mark.parametrize("scale", [2.0 ** 60, -2.0 ** 60])
def test_the_largest_scales(cuda_device, cus, E, scale):
    """Rows without experts have weights of 0, and no weight that is a number becomes another."""
    x = torch.randn(70, E, generator=synth.make_generator(8, cuda_device), device=cuda_device)
    x[::2] = -float("inf")
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids, w = fg.moe_route(x, 3, scoring=scoring, renormalize=renormalize, scale=scale)
            ri, rw, _ = mo.route(f64(x), 3, None, scoring, renormalize=renormalize, scale=scale)
            assert np.array_equal(ids.cpu().numpy(), ri) and bool((w[::2] == 0).all())
            assert np.all(np.abs(f64(w) - rw) <= 2.0 ** -16 * np.abs(rw))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups", [(16, 1, 1), (32, 1, 1), (32, 4, 2), (64, 1, 1), (160, 8, 3), (256, 1, 1), (256, 8, 4)])
def test_a_row_alone_and_among_many(cuda_device, E, groups, top_groups, scoring):
    """The same experts; weights that differ by the order of their sums at most. With u = 2^-24, of equal
    exponentials and sigmoids: a softmax's total is off by up to 20 u, its reciprocal and product
    by 2, the chosen scores' sum by 7, quotient and product by 2, on either side: below 64 u."""
    g = synth.make_generator(9, cuda_device)
    x = torch.randn(20000, E, generator=g, device=cuda_device)
    bias = torch.randn(E, generator=g, device=cuda_device) * 0.1
    bias[E // 2] = bias[0]
    x[:64, E // 2] = x[:64, 0]
    for b in (None, bias):
        for renormalize in (True, False):
            kw = dict(bias=b, scoring=scoring, groups=groups, top_groups=top_groups, group_best=2, renormalize=renormalize)
            ids, w = fg.moe_route(x, 5, **kw)
            again = fg.moe_route(x, 5, **kw)
            assert torch.equal(again[0], ids) and torch.equal(again[1], w)
            for n in (1, 50):
                few, wf = fg.moe_route(x[:n], 5, **kw)
                assert torch.equal(few, ids[:n]) and torch.equal(fg.moe_route(x[:n], 5, **kw)[1], wf)
                assert bool(((wf.double() - w[:n].double()).abs() <= 64 * 2.0 ** -24 * wf.double()).all())
                fg.set_num_cus(1)
                try:
                    one, w1 = fg.moe_route(x[:n], 5, **kw)
                finally:
                    fg.set_num_cus(0)
                assert torch.equal(one, few)
                assert bool(((wf.double() - w1.double()).abs() <= 64 * 2.0 ** -24 * wf.double()).all())
