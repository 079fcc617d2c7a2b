"""Sequences longer than their rows of the block table: slots past the table do not exist, and
everything else stays where it is. A narrow table acts as one whose further entries name no
page, which is what the oracle is given. Bounds as in the parity tests of the two operators."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp32_amd as fg
import test_gpu_paged_append as append
import test_gpu_paged_attention as attention

pytestmark = pytest.mark.gpu


def narrowed(setup, pages):
    setup.table = setup.table[:, :pages].contiguous()
    setup.pages = [row[:pages] + [-1] * (len(row) - pages) for row in setup.pages]
    return setup


@pytest.mark.parametrize("new", [1, 3])
def test_tokens_past_a_full_table_leave_the_cache_alone(cuda_device, new):
    """The first token past the last slot (and those after it) change no byte; their queries
    turn by the slots that they would have had."""
    s = narrowed(append.Setup(cuda_device, [new, 1], [48 + new, 5], 2, 2, 128, 16, seed=40), 3)
    rot = append.table_of(64, 64, cuda_device)
    out = s.run(rot)
    for page in s.pages[0][:3]:
        for now, before in zip(s.cache, s.before):
            assert torch.equal(now[page], before[page])
    s.check(out, rot)


CASES = [  # new tokens, lengths, pages of the table, Hq, Hkv, D, P
    ([20], [20], 1, 1, 1, 64, 16),
    ([20, 1, 7], [20, 33, 40], 2, 4, 2, 128, 16),
    ([130, 300], [200, 300], 1, 2, 2, 64, 128),
    ([40] * 30, [40 + i for i in range(30)], 2, 2, 2, 64, 32),
    ([5, 2], [400, 1], 2, 8, 1, 256, 64),               # all past the table
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,lens,pages,Hq,Hkv,D,P", CASES)
def test_tokens_that_fit_are_stored_in_their_own_slots(cuda_device, new, lens, pages, Hq, Hkv, D, P, interleaved):
    s = narrowed(append.Setup(cuda_device, new, lens, Hq, Hkv, D, P, seed=41), pages)
    rot = append.table_of(max(lens), D // 2, cuda_device)
    s.check(s.run(rot, interleaved), rot, interleaved)


@pytest.fixture(scope="module")
def workspace():
    return fg.make_attention_workspace()


ATTENTION = [  # new tokens, lengths, pages of the table, Hq, Hkv, D, P
    ([1, 1], [40, 100], 3, 4, 2, 128, 16),
    ([60, 7], [90, 50], 2, 6, 2, 64, 32),
    ([200], [333], 2, 4, 1, 128, 128),                  # rows on both sides of the table's end
    ([1] * 70, [20 + 13 * i % 97 for i in range(70)], 4, 2, 1, 64, 16),
    ([90], [1500], 10, 4, 2, 256, 64),
]


@pytest.mark.parametrize("window", [0, 1, 50, 700])
@pytest.mark.parametrize("new,lens,pages,Hq,Hkv,D,P", ATTENTION)
def test_rows_past_the_table_keep_their_positions(cuda_device, workspace, new, lens, pages, Hq, Hkv, D, P, window):
    s = narrowed(attention.Setup(cuda_device, new, lens, Hq, Hkv, D, P, seed=42), pages)
    ref = s.reference(window)
    s.check(*s.run(window=window, workspace=workspace), window, ref)
    s.check(*s.run(window=window), window, ref)
    assert int(workspace[: 64 << 10].count_nonzero()) == 0


def test_lengths_of_31_bits(cuda_device, workspace):
    """The largest length that the array holds: every slot of the table is before the rows."""
    s = attention.Setup(cuda_device, [2, 1], [64, 30], 2, 1, 64, 32, seed=43, poison=False)
    want, wl = s.run(workspace=workspace)
    lens = torch.tensor([2 ** 31 - 1, 30], dtype=torch.int32, device=cuda_device)
    wide = fg.paged_attention(s.q, s.cache, s.table[:, :2].contiguous(), lens, s.cu_q, workspace=workspace)
    assert torch.equal(wide[1], want[1]) and torch.equal(wide[2], want[2])  # the last row of 64 sees all 64 keys, too
    none = fg.paged_attention(s.q, s.cache, s.table[:, :2].contiguous(), lens, s.cu_q, window=100, workspace=workspace)
    assert bool((none[:2] == 0).all()) and torch.equal(none[2], want[2])
    t = append.Setup(cuda_device, [2, 1], [64, 30], 2, 1, 64, 32, seed=44)
    before = [x.clone() for x in t.cache]
    fg.rope_append_paged_kv(None, t.k[:2], t.v[:2], None, t.cache, t.table[:1, :2].contiguous(), lens[:1], t.cu_q[:2].contiguous())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(t.cache, before))
    assert np.all(append.f64(t.cache.k_scale) == append.f64(before[1]))
