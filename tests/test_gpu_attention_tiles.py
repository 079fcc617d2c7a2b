"""The attention's tiles of 48 and 64 rows, which a call takes when its rows are many enough to
give every compute unit a tile: here with few compute units, so that small calls take them.
Bounds as in the parity tests of attention."""
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
from test_gpu_paged_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[2, 12])
def few_cus(request):
    fg.set_num_cus(request.param)
    yield request.param
    fg.set_num_cus(0)


@pytest.fixture(scope="module")
def workspace():
    return fg.make_attention_workspace()


def takes_large_tiles(s, cus):
    """The host's rule, for the tests' own check that they reach what they are about."""
    rows = -(-s.T * (s.Hq // s.Hkv) // len(s.lens))
    most = 64 if s.D == 64 else 48
    tiles = -(-rows // most)
    return rows > 32 and tiles * most * 0.9 < -(-rows // 32) * 32 and tiles * len(s.lens) * s.Hkv >= cus


CASES = [  # new tokens, lengths, Hq, Hkv, P: 189 or 192 rows a key head and sequence on average
    ([192], [192], 12, 12, 16),
    ([48, 48], [700, 48], 24, 6, 64),                     # 4 heads a key head
    ([1, 319, 0, 448], [900, 319, 70, 1030], 3, 3, 128),  # ragged; a last tile of few rows
    ([9, 20], [40, 3000], 26, 2, 256),                    # 13 heads a key head: tiles begin inside a token's heads
    ([384, 0], [1, 900], 12, 12, 32),                     # more new tokens than keys: rows that see nothing
]


@pytest.mark.parametrize("window", [0, 1, 50, 700])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens,Hq,Hkv,P", CASES)
def test_large_tiles(cuda_device, workspace, few_cus, new, lens, Hq, Hkv, P, D, window):
    s = Setup(cuda_device, new, lens, Hq, Hkv, D, P, seed=20)
    assert takes_large_tiles(s, few_cus)
    ref = s.reference(window)
    split = s.run(window=window, workspace=workspace)
    s.check(*split, window, ref)
    s.check(*s.run(window=window), window, ref)
    again = s.run(window=window, workspace=workspace)
    assert torch.equal(again[0], split[0]) and torch.equal(again[1], split[1])
    assert int(workspace[: 64 << 10].count_nonzero()) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8])
def test_a_bad_code_in_a_large_tile(cuda_device, workspace, few_cus, group, D):
    new = 512 // group
    for window in (0, 3):
        for which in (0, 2):
            clean = Setup(cuda_device, [new], [new + 50], 12 * group, 12, D, 32, seed=21)
            assert takes_large_tiles(clean, few_cus)
            want, wl = clean.run(window=window, workspace=workspace)
            bad = Setup(cuda_device, [new], [new + 50], 12 * group, 12, D, 32, seed=21)
            slot = 50 + new // 2
            bad.cache[which][bad.pages[0][slot // 32], 5, slot % 32, 33] = 0x7F
            got, gl = bad.run(window=window, workspace=workspace)
            first, last = new // 2, min(new, new // 2 + (window or new))
            sound = torch.ones(new, 12 * group, dtype=torch.bool)
            sound[first:last, 5 * group:6 * group] = False
            assert torch.equal(got[sound], want[sound]) and torch.equal(gl[sound], wl[sound])
            assert bool(got[~sound][:, 33].isnan().all())
