"""The ways in which attention cuts a call into units, on few compute units so that small calls
reach each: one unit for each compute unit, whole tiles, rounds of chunks; more sequences than
a wave has lanes; lengths that leave most of the grid without a unit. Bounds as in the parity
tests of attention."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from test_gpu_paged_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def workspace():
    return fg.make_attention_workspace()


def ragged(n, most):
    return [1 + (most - 1) * (i * 37 % n) // n for i in range(n)]


CASES = [  # new tokens, lengths, Hq, Hkv, D, P
    ([1] * 70, ragged(70, 2600), 2, 1, 64, 64),        # over 64 sequences: counted in two passes
    ([1] * 70, [700] * 70, 1, 1, 128, 16),             # equal ones
    ([1] * 130, ragged(130, 900), 4, 2, 64, 32),
    ([1, 3, 1], [9000, 4100, 5], 4, 1, 128, 128),      # few tiles, long
    ([1] * 9, ragged(9, 6000), 8, 8, 128, 64),
    ([2, 1, 60, 1], [3000, 2999, 60, 0], 6, 2, 256, 32),
]


@pytest.mark.parametrize("window", [0, 600])
@pytest.mark.parametrize("cus", [1, 5, 40, 0])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D,P", CASES)
def test_every_cut_gives_the_same_rows(cuda_device, workspace, new, lens, Hq, Hkv, D, P, cus, window):
    s = Setup(cuda_device, new, lens, Hq, Hkv, D, P, seed=30)
    fg.set_num_cus(cus)
    try:
        out, lse = s.run(window=window, workspace=workspace)
        again = s.run(window=window, workspace=workspace)
    finally:
        fg.set_num_cus(0)
    s.check(out, lse, window)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert int(workspace[: 64 << 10].count_nonzero()) == 0


def test_a_table_far_wider_than_its_sequences(cuda_device, workspace):
    """The grid is sized for the table's width; the sequences are short."""
    s = Setup(cuda_device, [1, 2], [40, 300], 4, 2, 128, 16, seed=31)
    want = s.run(workspace=workspace)
    s.table = torch.cat([s.table, torch.full((2, 20000), -1, dtype=torch.int32, device=cuda_device)], dim=1)
    got = s.run(workspace=workspace)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert int(workspace[: 64 << 10].count_nonzero()) == 0
