"""Limits and promises of the layer operators that need no GPU to be checked."""
import glob
import os
import re

import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from test_layer_abi import APPEND, ATTEND, DEVICE, NULL, SHAPE, call


def test_attention_takes_tables_of_2_to_the_30_slots():
    """Key numbers are 32-bit, and a sequence of more keys would be cut where nothing may be."""
    for P, pages in ((16, 1 << 26), (64, 1 << 24), (256, 1 << 22)):
        assert call("fp8_paged_attention", ATTEND, P=P, max_pages=pages + 1, ld_bt=pages + 1) == SHAPE
        if not torch.cuda.is_available():  # the arguments are good and their addresses are not
            assert call("fp8_paged_attention", ATTEND, P=P, max_pages=pages, ld_bt=pages) == DEVICE


def test_what_is_no_gpu_tensor_is_refused_on_another_stream_as_well():
    x = torch.zeros(4, 256)
    for bad, error in ((7, TypeError), ([1.0], TypeError), (None, TypeError), (x, ValueError), (x[0], ValueError)):
        with pytest.raises(error):
            fg.rmsnorm_backward(bad, x, x[:, 0], x[0], stream=object())


def test_a_table_without_pages_may_have_no_address():
    for name, defaults in (("fp8_rope_append_paged_kv", APPEND), ("fp8_paged_attention", ATTEND)):
        assert call(name, defaults, block_table=None, max_pages=1, ld_bt=1) == NULL
        if not torch.cuda.is_available():
            assert call(name, defaults, block_table=None, max_pages=0, ld_bt=0) == DEVICE


def test_assembly_says_which_registers_it_writes():
    """m0 is the compiler's to use as well: a statement that sets it has to name it."""
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(fg.__file__), "csrc_layer", "*")):
        for statement in re.findall(r"\basm\b[^;]*?\((.*?)\);", open(path).read(), re.S):
            if re.search(r"s_mov_b32 m0,", statement):
                found += 1
                assert '"m0"' in statement.rsplit(":", 1)[1], (path, statement)
    assert found == 2


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_heads_are_less_than_2_to_the_31_columns(D):
    """A head's first column is a 32-bit number in the kernels."""
    for name, defaults, rows in (("fp8_rope_append_paged_kv", {**APPEND, "rot_dim": 0}, ("ldq", "ldqo")),
                                 ("fp8_paged_attention", ATTEND, ("ldq", "ldo"))):
        wide = dict.fromkeys(rows, 1 << 40)
        assert call(name, defaults, T=1, B=1, Hq=(1 << 31) // D, Hkv=2, D=D, **wide) == SHAPE
        if not torch.cuda.is_available():
            assert call(name, defaults, T=1, B=1, Hq=(1 << 31) // D - 2, Hkv=2, D=D, **{**wide, **({"ldk": 512, "ldv": 512} if "ldk" in defaults else {})}) == DEVICE
    assert call("fp8_rope_append_paged_kv", {**APPEND, "rot_dim": 0}, T=1, B=1, Hkv=(1 << 31) // D, D=D, ldk=1 << 40, ldv=1 << 40) == SHAPE
