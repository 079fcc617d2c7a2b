"""The limits that the header of the expert and head operators names: calls at them are taken, and
calls one past them are refused before anything is launched."""
import re

import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from test_moe_abi import DEVICE, DISPATCH, GATHER, HEADER, HEADS, HEADS_GRAD, ROUTE, ROUTE_GRAD, SHAPE, call

MOST = 2 ** 31 - 2 ** 18 - 1  # choices, rows, heads


@pytest.fixture
def without_a_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: valid calls would be launched")


def test_choices_rows_and_heads(without_a_gpu):
    assert {2 ** 31 - 2 ** int(n) - 1 for n in re.findall(r"below 2\^31 - 2\^(\d+)", open(HEADER).read())} == {MOST}
    workspace = dict(workspace_bytes=1 << 40)
    for T, top_k in ((MOST, 1), (MOST // 2, 2), (MOST // 64, 64)):
        kw = dict(T=T, top_k=top_k, ld_sa=-(-T // 4) * 4)
        assert call("fp8_moe_dispatch", DISPATCH, **kw, **workspace) == DEVICE
        assert call("fp8_moe_gather", GATHER, **kw) == DEVICE
        kw["T"], kw["ld_sa"] = T + 1, kw["ld_sa"] + 4
        assert call("fp8_moe_dispatch", DISPATCH, **kw, **workspace) == SHAPE
        assert call("fp8_moe_gather", GATHER, **kw) == SHAPE
    rows = MOST // 128 * 128
    for n, code in ((rows, DEVICE), (rows + 128, SHAPE)):
        assert call("fp8_moe_dispatch", DISPATCH, rows=n, ld_sax=n) == code
        assert call("fp8_moe_gather", GATHER, rows=n, ld_sax=n) == code
    for T, Hq, Hk in ((MOST, 1, 0), (MOST // 3, 2, 1), (1, 1 << 23, 1 << 23)):
        kw = dict(T=T, Hq=Hq, Hk=Hk, ldq=max(Hq, 1) * 128, ldk=max(Hk, 1) * 128)
        out, grad = dict(ldqo=kw["ldq"], ldko=kw["ldk"]), dict(lddq=kw["ldq"], lddk=kw["ldk"], lddqo=kw["ldq"], lddko=kw["ldk"])
        assert call("fp8_qk_norm_rope", HEADS, **kw, **out) == DEVICE
        assert call("fp8_qk_norm_rope_backward", HEADS_GRAD, **kw, **grad) == DEVICE
        kw["T"] = MOST // (Hq + Hk) + 1
        assert call("fp8_qk_norm_rope", HEADS, **kw, **out) == SHAPE
        assert call("fp8_qk_norm_rope_backward", HEADS_GRAD, **kw, **grad) == SHAPE


def test_scales(without_a_gpu):
    """Up to 2^60: over 1e-20, what a row without experts is scaled by, that is a number."""
    for name, defaults in (("fp8_moe_route", ROUTE), ("fp8_moe_route_backward", ROUTE_GRAD)):
        for scale in (2.0 ** 60, -2.0 ** 60, 0.0):
            assert call(name, defaults, scale=scale) == DEVICE
        for scale in (2.0 ** 61, -2.0 ** 61, 1e30, float("inf")):
            assert call(name, defaults, scale=scale) == SHAPE


def test_rows_of_no_tokens_are_refused_where_those_of_one_are():
    assert fg.moe_rows(0, 64, 1024) == 0 and fg.make_moe_layout(0, 64, 1024, device="cpu").sources.shape == (0,)
    for top_k, experts in ((0, 8), (65, 8), (2, 0), (2, 1025)):
        for tokens in (0, 1):
            with pytest.raises(ValueError):
                fg.moe_rows(tokens, top_k, experts)
            with pytest.raises(ValueError):
                fg.make_moe_layout(tokens, top_k, experts, device="cpu")
