"""Limits and promises of the layer operators that need no GPU to be checked."""
import torch

from test_layer_abi import ATTEND, DEVICE, SHAPE, call


def test_attention_takes_tables_of_2_to_the_30_slots():
    """Key numbers are 32-bit, and a sequence of more keys would be cut where nothing may be."""
    for P, pages in ((16, 1 << 26), (64, 1 << 24), (256, 1 << 22)):
        assert call("fp8_paged_attention", ATTEND, P=P, max_pages=pages + 1, ld_bt=pages + 1) == SHAPE
        if not torch.cuda.is_available():  # the arguments are good and their addresses are not
            assert call("fp8_paged_attention", ATTEND, P=P, max_pages=pages, ld_bt=pages) == DEVICE
